// rms_norm.cu -- the root-mean-square norm's entry points (cns_rms_norm,
// cns_rms_norm_backward) and the join of the parts of the gain's gradient.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cns.h"
#include "cns_host.h"
#include "rms_norm_kernels.cuh"

namespace cns {
namespace {

constexpr int kJoinColumns = 8, kJoinRows = 64, kJoinHeld = 5;   // 8 columns: a sector of each part

// dgain = the sum of the parts.  A CTA has 8 columns, its 64 groups of 8 threads every 64th part, so that few columns
// have CTAs enough too and a thread's loads are in flight together: the gradient of 16384 x 1000 bf16 takes 26.8 us so,
// 27.4 with 32 columns and 32 groups or with 32 groups of 8; of 777 x 1000 f32 4.55, 4.61 and 4.61.
__global__ void __launch_bounds__(kJoinColumns * kJoinRows)
join_parts_kernel(const float *parts, int count, int width, float *dgain)
{
    __shared__ float s_sum[kJoinRows * kJoinColumns / 32][kJoinColumns];
    const int column = threadIdx.x % kJoinColumns, e = blockIdx.x * kJoinColumns + column;
    grid_dependency_wait();
    float sum = 0.f;
    for (int i = threadIdx.x / kJoinColumns; i < count; i += kJoinRows * kJoinHeld) {
        float v[kJoinHeld];
#pragma unroll
        for (int k = 0; k < kJoinHeld; ++k)
            v[k] = i + k * kJoinRows < count && e < width ? parts[static_cast<int64_t>(i + k * kJoinRows) * width + e] : 0.f;
#pragma unroll
        for (int k = 0; k < kJoinHeld; ++k)
            sum += v[k];
    }
#pragma unroll
    for (int d = kJoinColumns; d < 32; d *= 2)
        sum += __shfl_xor_sync(kFullWarp, sum, d);
    if (threadIdx.x % 32 < kJoinColumns)
        s_sum[threadIdx.x / 32][column] = sum;
    __syncthreads();
    if (threadIdx.x < kJoinColumns && e < width) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinRows * kJoinColumns / 32; ++i)
            sum += s_sum[i][column];
        dgain[e] = sum;
    }
}

bool type_ok(int32_t dtype) { return dtype >= CNS_DT_F32 && dtype <= CNS_DT_F16; }

int64_t bytes_of(int32_t dtype) { return dtype == CNS_DT_F32 ? 4 : 2; }

bool off(const void *p, int64_t bytes) { return address(p) % bytes != 0; }

// A matrix's stride (`packed` where it is 0); false if it is out of range.
bool stride_ok(int64_t given, int64_t packed, int64_t *stride)
{
    *stride = given ? given : packed;
    return *stride >= packed && *stride <= CNS_ROWS_MAX_STRIDE;
}

}  // namespace
}  // namespace cns

using namespace cns;

extern "C" int cns_rms_norm(const cns_rms_norm_t *n)
{
    TraceRange tr("cns_rms_norm", n ? static_cast<uint64_t>(n->rows) : 0);
    if (!n)
        return CNS_ERR_NULL_PTR;
    if (n->rows < 0 || n->rows > 0x7fffffff || n->width < 1 || n->width > CNS_NORM_MAX_WIDTH || !type_ok(n->dtype) ||
        !type_ok(n->gain_dtype) || (n->scale_block != 0 && n->scale_block != 32 && n->scale_block != 64 && n->scale_block != 128) ||
        (n->scale_type != CNS_SCALE_F32 && n->scale_type != CNS_SCALE_E8M0) || !std::isfinite(n->eps) || n->eps < 0.f)
        return CNS_ERR_INVALID_VALUE;
    const int64_t blocks = n->scale_block ? (n->width + n->scale_block - 1) / n->scale_block : 1;
    NormParams p = {};
    if (!stride_ok(n->x_stride, n->width, &p.x_stride) || !stride_ok(n->residual_stride, n->width, &p.residual_stride) ||
        !stride_ok(n->h_stride, n->width, &p.h_stride) || !stride_ok(n->y_stride, n->width, &p.y_stride) ||
        !stride_ok(n->q_stride, n->width, &p.q_stride) || !stride_ok(n->scales_stride, blocks, &p.scales_stride))
        return CNS_ERR_INVALID_VALUE;
    if ((n->h_dev && !n->residual_dev) || (n->scales_dev && !n->q_dev))
        return CNS_ERR_INVALID_VALUE;
    if (n->rows > 0 && (!n->x_dev || (!n->y_dev && !n->q_dev) || (n->residual_dev && !n->h_dev) || (n->q_dev && !n->scales_dev)))
        return CNS_ERR_NULL_PTR;
    const int64_t e = bytes_of(n->dtype);
    if (off(n->x_dev, e) || off(n->residual_dev, e) || off(n->h_dev, e) || off(n->y_dev, e) ||
        off(n->gain_dev, bytes_of(n->gain_dtype)) || (n->scale_type == CNS_SCALE_F32 && off(n->scales_dev, 4)))
        return CNS_ERR_INVALID_VALUE;
    if ((n->y_dev && (n->y_dev == n->x_dev || n->y_dev == n->residual_dev || n->y_dev == n->h_dev)) ||
        (n->h_dev && ((n->h_dev == n->x_dev && p.h_stride != p.x_stride) ||
                      (n->h_dev == n->residual_dev && p.h_stride != p.residual_stride))))
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    if (n->rows == 0)
        return CNS_SUCCESS;
    p.x = n->x_dev;
    p.residual = n->residual_dev;
    p.gain = n->gain_dev;
    p.h = n->h_dev;
    p.y = n->y_dev;
    p.q = n->q_dev;
    p.scales = n->scales_dev;
    p.rows = n->rows;
    p.width = n->width;
    p.gain_dtype = n->gain_dtype;
    p.block = n->scale_block;
    p.power = n->scale_type == CNS_SCALE_E8M0;
    p.eps = n->eps;
    uint64_t bits = address(p.x) | address(p.gain) | (p.x_stride * e) | (n->width * e);
    if (p.residual)
        bits |= address(p.residual) | (p.residual_stride * e) | address(p.h) | (p.h_stride * e);
    if (p.y)
        bits |= address(p.y) | (p.y_stride * e);
    if (p.q)
        bits |= (address(p.q) | p.q_stride) * e;   // a vector's elements, in 8 bits
    const bool wide = bits % 16 == 0;
    cudaStream_t s = to_stream(n->stream);
    CNS_CUDA(n->dtype == CNS_DT_F32    ? launch_rms_norm_f32(p, wide, dev.sm_count, s)
             : n->dtype == CNS_DT_BF16 ? launch_rms_norm_bf16(p, wide, dev.sm_count, s)
                                       : launch_rms_norm_f16(p, wide, dev.sm_count, s));
    return CNS_SUCCESS;
}

extern "C" int cns_rms_norm_workspace_bytes(int64_t rows, int32_t width, size_t *bytes)
{
    if (!bytes)
        return CNS_ERR_NULL_PTR;
    if (rows < 0 || rows > 0x7fffffff || width < 1 || width > CNS_NORM_MAX_WIDTH)
        return CNS_ERR_INVALID_VALUE;
    *bytes = sizeof(float) * static_cast<size_t>(rows < kNormMaxParts ? rows : kNormMaxParts) * static_cast<size_t>(width);
    return CNS_SUCCESS;
}

extern "C" int cns_rms_norm_backward(const cns_rms_norm_grad_t *n)
{
    TraceRange tr("cns_rms_norm_backward", n ? static_cast<uint64_t>(n->rows) : 0);
    if (!n)
        return CNS_ERR_NULL_PTR;
    size_t need = 0;
    NormGradParams p = {};
    if (cns_rms_norm_workspace_bytes(n->rows, n->width, &need) || !type_ok(n->dtype) || !type_ok(n->gain_dtype) ||
        !std::isfinite(n->eps) || n->eps < 0.f || !stride_ok(n->h_stride, n->width, &p.h_stride) ||
        !stride_ok(n->dy_stride, n->width, &p.dy_stride) || !stride_ok(n->dh_stride, n->width, &p.dh_stride) ||
        !stride_ok(n->dx_stride, n->width, &p.dx_stride))
        return CNS_ERR_INVALID_VALUE;
    if (n->rows > 0 && (!n->h_dev || !n->dy_dev || !n->dx_dev || (n->dgain_dev && !n->workspace_dev)))
        return CNS_ERR_NULL_PTR;
    const int64_t e = bytes_of(n->dtype);
    if (off(n->h_dev, e) || off(n->dy_dev, e) || off(n->dh_dev, e) || off(n->dx_dev, e) || off(n->dgain_dev, 4) ||
        off(n->gain_dev, bytes_of(n->gain_dtype)) || off(n->workspace_dev, 16) || (n->dgain_dev && n->workspace_bytes < need))
        return CNS_ERR_INVALID_VALUE;
    if (n->dx_dev && (n->dx_dev == n->h_dev || (n->dx_dev == n->dy_dev && p.dx_stride != p.dy_stride) ||
                      (n->dx_dev == n->dh_dev && p.dx_stride != p.dh_stride)))
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    p.h = n->h_dev;
    p.gain = n->gain_dev;
    p.dy = n->dy_dev;
    p.dh = n->dh_dev;
    p.dx = n->dx_dev;
    p.dgain = n->dgain_dev;
    p.parts = static_cast<float *>(n->workspace_dev);
    p.rows = n->rows;
    p.width = n->width;
    p.gain_dtype = n->gain_dtype;
    p.eps = n->eps;
    cudaStream_t s = to_stream(n->stream);
    int parts = 0;
    if (n->rows > 0) {
        uint64_t bits = address(p.h) | address(p.gain) | address(p.dy) | address(p.dx) | (p.h_stride * e) | (p.dy_stride * e) |
                        (p.dx_stride * e) | (n->width * e);
        if (p.dh)
            bits |= address(p.dh) | (p.dh_stride * e);
        const bool wide = bits % 16 == 0;
        CNS_CUDA(n->dtype == CNS_DT_F32    ? launch_rms_norm_backward_f32(p, wide, dev.sm_count, &parts, s)
                 : n->dtype == CNS_DT_BF16 ? launch_rms_norm_backward_bf16(p, wide, dev.sm_count, &parts, s)
                                           : launch_rms_norm_backward_f16(p, wide, dev.sm_count, &parts, s));
    }
    if (!n->dgain_dev || parts == 1)   // the only part is dgain
        return CNS_SUCCESS;
    cudaLaunchAttribute early;
    cudaLaunchConfig_t cfg = early_launch(&early);
    cfg.gridDim = dim3((n->width + kJoinColumns - 1) / kJoinColumns);
    cfg.blockDim = dim3(kJoinColumns * kJoinRows);
    cfg.stream = s;
    CNS_CUDA(cudaLaunchKernelEx(&cfg, join_parts_kernel, static_cast<const float *>(p.parts), parts, n->width, n->dgain_dev));
    return CNS_SUCCESS;
}
