// kda_sums.hip -- sums of the columns of a matrix of partial sums, in a fixed order: what the
// gradients of weights, biases and scales are finished with; and a fill or copy for batches that
// hold no row (a kernel, so that a caller may capture the call in a graph).
#include "kda_rows.h"

namespace kda {
namespace {

// 16 groups of rows for 64 columns: a column's rows are read by 16 threads, each in order, and
// the 16 sums are added in order.
__global__ __launch_bounds__(1024) void column_sums_kernel(const ColumnSums a) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, group = threadIdx.x / 64;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < a.cols) {
#pragma unroll 8
        for (int r = group; r < a.rows; r += 16) s += a.x[(int64_t)r * a.cols + c];
    }
    part[group][lane] = s;
    __syncthreads();
    if (group == 0 && c < a.cols) {
        for (int g = 1; g < 16; ++g) s += part[g][lane];
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
    hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)(((int64_t)a.cols + 63) / 64)), dim3(1024), 0, stream, a);
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
