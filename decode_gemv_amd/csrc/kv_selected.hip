// kv_selected.hip -- attention of new tokens over pages that were chosen for
// each of them and each kv head (kv_select.hip): the kernel of kv_rows.hpp, a
// row tile being the query heads of one token and kv head.  Pages come in the
// order of their positions and the row's own is the last, so that what a row
// sees is one run of tokens from 0 on, without a mask.
//
// 16 rows of up to 2048 tokens, 32 heads on 8 of 128 (36 MB): 13.7 us (kernel trace),
// 2.6 TB/s, and 3.9 to join the chunks.  A wavefront has only four steps of 32 tokens: the chain
// of loads before the first key (the selection, then its pages) takes 1.8 us, the
// meeting of the wavefronts is another wait, and in between a step's unpacking
// takes as long as its memory.  Sixteen wavefronts a workgroup, chunks half and
// twice as long, and the entries or the queries loaded before the selection's
// lengths measured the same or worse, eight wavefronts too but for heads of 256,
// where they took 33.9 us and not 35.8 of 100 workgroups of 1536 tokens in two
// chunks each, and 42.9 and not 36.5 in six (with bounds, choice and join).
#include "kv_rows.hpp"

namespace {

template <int D, int ROWS, class T>
hipError_t launch(const KvAttend &a, hipStream_t s)
{
    const unsigned y = (unsigned)std::min(a.pieces, 1 << 15), z = (a.pieces + y - 1) / y;
    hipLaunchKernelGGL((k_kv_attend<D, ROWS, T, true>), dim3(a.g.kv_heads, y, z), dim3(NW * 64), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    return launch_join<D, ROWS, T, true>(a, a.pieces / a.splits, a.splits, s);
}

template <int D>
hipError_t launch_dim(const KvAttend &a, int dtype, int tile, hipStream_t s)
{
    if (tile == 8) return dtype == LW_F16 ? launch<D, 8, _Float16>(a, s) : launch<D, 8, __bf16>(a, s);
    return dtype == LW_F16 ? launch<D, 16, _Float16>(a, s) : launch<D, 16, __bf16>(a, s);
}

}  // namespace

hipError_t lw_launch_kv_selected(const KvAttend &a, int head_dim, int dtype, int tile, hipStream_t s)
{
    if (head_dim == 64) return launch_dim<64>(a, dtype, tile, s);
    if (head_dim == 128) return launch_dim<128>(a, dtype, tile, s);
    if (head_dim == 256) return launch_dim<256>(a, dtype, tile, s);
    return hipErrorInvalidValue;
}
