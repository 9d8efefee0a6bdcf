// kda_sums.hip -- sums of the columns of a matrix of partial sums, in a fixed order: what the
// gradients of weights, biases and scales are finished with; and a fill or copy for batches that
// hold no row (a kernel, so that a caller may capture the call in a graph).
#include "kda_rows.h"

namespace kda {
namespace {

// 1024 / C groups of rows for C columns: a column's rows are read by as many threads, each in order and
// 16 at a time, and their sums are added in order.  64 columns where there are many of them (256 rows of 20480
// columns: 5 us, with 32 columns 10), 32 where there are few and the rows' way is what it takes.
template <int SUM_C>
__global__ __launch_bounds__(1024) void column_sums_kernel(const ColumnSums a) {
    constexpr int SUM_G = 1024 / SUM_C;
    __shared__ float part[SUM_G][SUM_C];
    const int lane = threadIdx.x % SUM_C, group = threadIdx.x / SUM_C;
    const int64_t c = (int64_t)blockIdx.x * SUM_C + lane;
    float s = 0.f;
    if (c < a.cols) {
#pragma unroll 16
        for (int r = group; r < a.rows; r += SUM_G) s += a.x[(int64_t)r * a.cols + c];
    }
    part[group][lane] = s;
    __syncthreads();
    if (group == 0 && c < a.cols) {
#pragma unroll
        for (int g = 1; g < SUM_G; ++g) s += part[g][lane];
        const int64_t n = (int64_t)a.D * a.W;
        if (c < n) {
            if (a.first) a.first[c % a.D * a.W + c / a.D] = s;
        } else if (a.second) {
            a.second[c - n] = s;
        }
    }
}

__global__ __launch_bounds__(256) void fill_bytes_kernel(uint16_t *dst, const uint16_t *src, int64_t n) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) dst[i] = src ? src[i] : 0;
}

}  // namespace

hipError_t launch_column_sums(const ColumnSums &a, hipStream_t stream) {
    if (a.cols <= 0) return hipSuccess;
    if (a.cols >= 8192) hipLaunchKernelGGL(column_sums_kernel<64>, dim3((unsigned)(((int64_t)a.cols + 63) / 64)), dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL(column_sums_kernel<32>, dim3((unsigned)((a.cols + 31) / 32)), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_fill_bytes(void *dst, const void *src, int64_t bytes, hipStream_t stream) {
    const int64_t n = bytes / 2, blocks = (n + 255) / 256;
    if (n <= 0) return hipSuccess;
    hipLaunchKernelGGL(fill_bytes_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, static_cast<uint16_t *>(dst),
                       static_cast<const uint16_t *>(src), n);
    return hipGetLastError();
}

}  // namespace kda
