// Sums of many blocks' partial rows: the last step of the gradients of parameters that every token shares.
#include "gla_internal.h"

namespace gla {
namespace {

__device__ __forceinline__ void store(const ColumnOuts& out, long long i, float s)
{
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (i >= 0 && i < out.o[k].n && out.o[k].to) out.o[k].to[i] = s;
        i -= out.o[k].n;
    }
}

// 32 columns per block; a column's rows are taken 32 apart, then over the 32.
__global__ void __launch_bounds__(1024) gla_column_sum_kernel(const float* part, long long rows, long long cols, ColumnOuts out)
{
    __shared__ float red[32][33];
    const long long i = (long long)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (i < cols)
        for (long long r = threadIdx.y; r < rows; r += 32) s += part[r * cols + i];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || i >= cols) return;
    s = 0.f;
    for (int k = 0; k < 32; ++k) s += red[k][threadIdx.x];
    store(out, i, s);
}

// Few rows: a thread per column (4 rows of 73728 columns: 11 us in blocks of 32, 3 so).
__global__ void __launch_bounds__(256) gla_column_sum_few_kernel(const float* part, long long rows, long long cols, ColumnOuts out)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= cols) return;
    float s = 0.f;
#pragma unroll 4
    for (long long r = 0; r < rows; ++r) s += part[r * cols + i];
    store(out, i, s);
}

}  // namespace

cudaError_t launch_column_sum(const float* part, long long rows, long long cols, const ColumnOuts& out, cudaStream_t s)
{
    if (rows <= 16) gla_column_sum_few_kernel<<<(unsigned)((cols + 255) / 256), 256, 0, s>>>(part, rows, cols, out);
    else gla_column_sum_kernel<<<(unsigned)((cols + 31) / 32), dim3(32, 32), 0, s>>>(part, rows, cols, out);
    return cudaGetLastError();
}

}  // namespace gla
