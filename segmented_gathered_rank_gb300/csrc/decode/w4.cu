// Matrix products with 4-bit weights (lora_w4_matvec):
//   y[t][n] = sum_g s[n][g] * sum_{k in g} x[t][k] * (c[n][k] - z[n][g])
#include "decode.cuh"

namespace lora {
namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 8;

// One warp per output row and 8 tokens; each lane takes 8 codes at a time.
template <typename E>
__global__ void __launch_bounds__(kWarps * 32) w4_kernel(const E *__restrict__ x, int T, int h_in,
                                                        const uint8_t *__restrict__ codes,
                                                        const __nv_bfloat16 *__restrict__ scales,
                                                        const uint8_t *__restrict__ zeros, int group_shift, int h_out,
                                                        E *__restrict__ y) {
    const int n = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t0 = blockIdx.y * kTokens, nt = min(kTokens, T - t0);
    if (n >= h_out) return;
    const long long groups = h_in >> group_shift;
    float acc[kTokens] = {};
    for (int k = lane * 8; k < h_in; k += 256) {
        const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + ((long long)n * h_in + k) / 2);
        const long long g = n * groups + (k >> group_shift);
        const float s = __bfloat162float(scales[g]);
        const float z = zeros ? (float)zeros[g] : 8.f;
        for (int t = 0; t < nt; ++t) {
            float xs[8], part = 0.f;
            load8(x + (long long)(t0 + t) * h_in + k, xs);
#pragma unroll
            for (int e = 0; e < 8; ++e) part += xs[e] * ((float)((c >> (4 * e)) & 15u) - z);
            acc[t] += s * part;
        }
    }
    for (int t = 0; t < nt; ++t) {
        const float a = warp_sum(acc[t]);
        if (lane == 0) {
            if constexpr (sizeof(E) == 2) y[(long long)(t0 + t) * h_out + n] = __float2bfloat16_rn(a);
            else y[(long long)(t0 + t) * h_out + n] = a;
        }
    }
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_w4_matvec(int dtype, const void *x, int T, int h_in, const void *codes, const void *scales,
                              const void *zeros, int group, int h_out, void *y, lora_stream stream) {
    if ((dtype != LORA_F32 && dtype != LORA_BF16) || T < 0 || h_in <= 0 || h_out <= 0) return LORA_ERR_ARG;
    if ((group != 32 && group != 64 && group != 128) || h_in % group) return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!x || !codes || !scales || !y || !aligned16(x) || !aligned16(codes) || !aligned16(y) ||
        ((uintptr_t)scales & 1u))
        return LORA_ERR_ARG;
    const int shift = group == 32 ? 5 : group == 64 ? 6 : 7;
    const dim3 grid((h_out + kWarps - 1) / kWarps, (T + kTokens - 1) / kTokens);
    if (grid.y > 65535) return LORA_ERR_SHAPE;
    cudaStream_t st = (cudaStream_t)stream;
    const uint8_t *c = static_cast<const uint8_t *>(codes), *z = static_cast<const uint8_t *>(zeros);
    const __nv_bfloat16 *s = static_cast<const __nv_bfloat16 *>(scales);
    if (dtype == LORA_BF16)
        w4_kernel<<<grid, kWarps * 32, 0, st>>>(static_cast<const __nv_bfloat16 *>(x), T, h_in, c, s, z, shift, h_out,
                                                static_cast<__nv_bfloat16 *>(y));
    else
        w4_kernel<<<grid, kWarps * 32, 0, st>>>(static_cast<const float *>(x), T, h_in, c, s, z, shift, h_out,
                                                static_cast<float *>(y));
    count_launch();
    return cuda_status(cudaGetLastError());
}
