// Prints "lanes, channels of a head, head of the warp, word of it, its place" for every width that a warp's exchange buffer
// serves, and before them the buffer's words.
#include <cstdio>

#include "norm_exchange.h"

template <int kLanes>
void places(int from, int to)
{
    for (int dim = from; dim <= to; dim += 8)
        for (int sub = 0; sub < 32 / kLanes; ++sub)
            for (int c = 0; c < dim; c += 2)
                std::printf("%d %d %d %d %d\n", kLanes, dim, sub, c / 2, h3fp4::exchange_at<kLanes>(sub, c));
}

int main()
{
    std::printf("%d\n", h3fp4::kExchangeWords);
    places<4>(8, 64);
    places<8>(72, 128);
    places<16>(136, 256);
}
