// Attention of several query rows over a cache of bf16 rows (bitq_rows.h).
#include "bitq_rows.h"

namespace bitq {

template <int NC, bool Q32>
static void launch_rows(const RowsArgs& a, int rw, unsigned grid, hipStream_t st) {
    const dim3 block(64 * rows_waves(rw));
    if (rw == 4) hipLaunchKernelGGL((rows_attn_kernel<BITQ_KV_BF16, NC, Q32, 4>), dim3(grid), block, 0, st, a);
    else hipLaunchKernelGGL((rows_attn_kernel<BITQ_KV_BF16, NC, Q32, 1>), dim3(grid), block, 0, st, a);
}

template <bool Q32>
static void launch_rows_dim(const RowsArgs& a, int nc, int rw, unsigned grid, hipStream_t st) {
    switch (nc) {
        case 1: launch_rows<1, Q32>(a, rw, grid, st); break;
        case 2: launch_rows<2, Q32>(a, rw, grid, st); break;
        case 3: launch_rows<3, Q32>(a, rw, grid, st); break;
        case 4: launch_rows<4, Q32>(a, rw, grid, st); break;
        case 5: launch_rows<5, Q32>(a, rw, grid, st); break;
        case 6: launch_rows<6, Q32>(a, rw, grid, st); break;
        case 7: launch_rows<7, Q32>(a, rw, grid, st); break;
        default: launch_rows<8, Q32>(a, rw, grid, st); break;
    }
}

void launch_rows_bf16(const RowsArgs& a, int nc, bool q32, int rw, unsigned grid, void* stream) {
    if (q32) launch_rows_dim<true>(a, nc, rw, grid, static_cast<hipStream_t>(stream));
    else launch_rows_dim<false>(a, nc, rw, grid, static_cast<hipStream_t>(stream));
}

}  // namespace bitq
