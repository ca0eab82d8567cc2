// Host-side helpers shared by the entry points: argument checks, the device status word
// and TMA tensor-map encoding.  No allocation; the only state is a per-device cache of
// the status word's address and of kernel attributes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "oasr_attn.h"

namespace oasr {

// Device address of the status word on the current device (nullptr on failure).
unsigned* status_word();

// Number of SMs of the current device (cached; 0 on failure).
int sm_count();

// Encode a 3-D bf16 tensor map over rows of [rows, H, 64] with a box of box_rows rows of
// one head, 128-byte swizzled.  Returns false if the driver rejects it.
bool encode_rows_bf16(CUtensorMap* map, const void* base, long long rows, int H, int box_rows);

// Encode a 4-D bf16 tensor map over the rows of [rows, H, 64] (rows a multiple of 8) viewed as
// {64, row % 8, head, row / 8}, with a box of two adjacent heads and box_rows rows (a multiple
// of 8), 128-byte swizzled: in shared memory a box is [row / 8][head][row % 8][64], so every
// 8 rows of one head form one 1 KB swizzle atom.  Returns false if the driver rejects it.
bool encode_head_pairs_bf16(CUtensorMap* map, const void* base, long long rows, int H, int box_rows);

// Encode a 2-D map over 64-byte rows (the 8-bit pools; an even number of them) with a box of box_rows
// rows, as 128-byte lines of two, 128-byte swizzled; its second coordinate counts lines.  Returns
// false if the driver rejects it.
bool encode_rows_e4m3(CUtensorMap* map, const void* base, long long rows, int box_rows);

// Encode a 2-D map over rows of row_bytes bytes (a multiple of 16) with a box of 64 bytes of box_rows rows,
// not swizzled or (swizzle64) with the 16-byte chunks of rows 2i and 2i + 1 exchanged by i % 4.  Returns false if
// the driver rejects it.
bool encode_bytes(CUtensorMap* map, const void* base, long long rows, int row_bytes, int box_rows, bool swizzle64 = false);

// Encode a 2-D map over rows of row_bytes bytes (a multiple of 16) with a box of 128 bytes of box_rows rows, 128-byte
// swizzled.  Returns false if the driver rejects it.
bool encode_bytes128(CUtensorMap* map, const void* base, long long rows, int row_bytes, int box_rows);

// Encode a 3-D bf16 map over rows of [rows, H, 64] that lie row_stride elements apart (a multiple of 8) with a box
// of box_heads heads of box_rows rows, 128-byte swizzled: in shared memory [row][head][64].  Returns false if the
// driver rejects it.
bool encode_head_rows_bf16(CUtensorMap* map, const void* base, long long rows, int H, long long row_stride, int box_heads,
                           int box_rows);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline oasr_status launch_status()
{
    return cudaGetLastError() == cudaSuccess ? OASR_OK : OASR_ERR_CUDA;
}

// Launch with programmatic stream serialization: the grid's CTAs may be scheduled while the
// previous grid on the stream drains.  Every kernel launched this way executes
// griddepcontrol.wait before its first global access, so it still sees all of the previous
// grid's writes.
template <typename... KArgs, typename... Args>
oasr_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem,
                       cudaStream_t stream, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...) != cudaSuccess)
        return OASR_ERR_CUDA;
    return launch_status();
}

// The same with clusters of `ctas` CTAs (the grid's x a multiple of it).
template <typename... KArgs, typename... Args>
oasr_status launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, int ctas,
                               cudaStream_t stream, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...) != cudaSuccess)
        return OASR_ERR_CUDA;
    return launch_status();
}

// Held while a kernel's attributes are changed: calls from several threads may want different ones.
inline std::mutex g_attribute_mutex;

// Raise the dynamic shared-memory limit of `func` on the current device to at least `bytes`; done: the limits
// set so far, by device.  They only ever rise, whatever the threads that call it at once want.
template <typename F>
bool ensure_smem(F* func, int bytes, int (&done)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE) >= bytes) return true;
    std::lock_guard<std::mutex> lock(g_attribute_mutex);
    if (done[dev] >= bytes) return true;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(func),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return false;
    __atomic_store_n(&done[dev], bytes, __ATOMIC_RELEASE);
    return true;
}

}  // namespace oasr
