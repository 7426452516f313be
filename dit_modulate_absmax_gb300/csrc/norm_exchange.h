// norm_exchange.h -- where the heads of a warp lie in its exchange buffer, for
// pairs of channels that neither lie side by side nor face each other (see
// norm_rope.cu).  Plain arithmetic, so that the host can enumerate it.
#pragma once

#ifdef __CUDACC__
#define H3FP4_HOST_DEVICE __host__ __device__
#else
#define H3FP4_HOST_DEVICE
#endif

namespace h3fp4 {

constexpr int kExchangeWords = 280;   // of a warp

// Word of a channel in the warp's exchange buffer: heads one after another, moved so that the lanes' words, four apart, fall
// into different banks.  At 16 lanes the words of a head are moved apart within it too, by 6 at most, which its room of 136
// words holds besides its 128.
template <int kLanes>
H3FP4_HOST_DEVICE constexpr int exchange_at(int sub, int channel)
{
    const int w = channel >> 1;
    return sub * (8 * kLanes + (kLanes == 16 ? 8 : 0)) + w + (kLanes == 16 ? 2 * (w >> 5) : 0) + (sub & 3) + (kLanes == 4 ? 16 * (sub >> 2) : 0);
}

}  // namespace h3fp4
