// kvtables.cuh -- launcher of the batch's tables.
#pragma once

#include "launch.h"

namespace h3fp4 {

cudaError_t launch_kv_tables(const h3fp4_kv_requests &q, cudaStream_t st);
cudaError_t read_kv_tables_error(uint32_t *code);

}  // namespace h3fp4
