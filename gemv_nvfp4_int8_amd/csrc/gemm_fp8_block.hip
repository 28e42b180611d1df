// gemm_fp8_block.hip -- block-scaled FP8 GEMM:
//
//   C[i,j] = bf16( sum_b as[i,b] * ws[j/128,b] * P_b[i,j] ),
//   P_b[i,j] = sum_{t in block b} e4m3(a[i,t]) * e4m3(w[j,t]),  128 K per block.
//
// P_b is formed on the matrix core in F32 from zero; as[i,b] * ws[j/128,b] is
// one F32 product per row and block, and acc += P_b * that one FMA per output
// and block on the vector ALU.
//
// The MFMAs compute C^T tiles (W fragment as the first operand): a lane then
// holds one row of C, so its scale is one value per lane and block and needs
// no broadcast.
#include "gemm_common.hpp"
#include "qp_launch.hpp"

namespace qp {
namespace {

constexpr int FB_T = 128, FB_BK = 128, FB_PITCH = FB_BK + 16;

__device__ __forceinline__ i32x8 frag32(const uint8_t *p)
{
    const i32x4 a = *reinterpret_cast<const i32x4 *>(p);
    const i32x4 b = *reinterpret_cast<const i32x4 *>(p + 16);
    return (i32x8){a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// 128 x 128 tiles, any shape: operand stages of one K block go through
// registers (zeros past the edges) into two LDS buffers.
__global__ __launch_bounds__(256) void k_fp8_gemm_block(
    const uint8_t *__restrict__ A, const float *__restrict__ as,
    const uint8_t *__restrict__ W, const float *__restrict__ ws,
    uint16_t *__restrict__ out, uint32_t M, uint32_t N, uint32_t K,
    uint32_t mtiles, uint32_t ntiles)
{
    __shared__ __attribute__((aligned(16))) uint8_t sA[2][FB_T * FB_PITCH];
    __shared__ __attribute__((aligned(16))) uint8_t sW[2][FB_T * FB_PITCH];

    uint32_t tm, tn;
    tile_coords(mtiles, ntiles, tm, tn);
    const uint32_t m0 = tm * FB_T, n0 = tn * FB_T;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave & 1, wn = wave >> 1;
    const uint32_t kb = (K + FB_BK - 1) / FB_BK;

    StageLoader<FB_T, FB_BK> la, lw;
    f32x16 acc[2][2] = {};

    // this lane's two rows of C and its tile's row of the weight's scale grid
    uint32_t row[2];
    const float *asr[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        row[t] = m0 + wm * 64 + 32 * t + (lane & 31);
        asr[t] = as + (size_t)min(row[t], M - 1) * kb;
    }
    const float *wsr = ws + (size_t)tn * kb;

    la.load(A, K, m0, M, 0, K);
    lw.load(W, K, n0, N, 0, K);
    la.store(sA[0]);
    lw.store(sW[0]);
    __syncthreads();

    const int arow = wm * 64 + (lane & 31), wrow = wn * 64 + (lane & 31);
    const int koff = 32 * (lane >> 5);
    for (uint32_t b = 0; b < kb; ++b) {
        const int buf = b & 1;
        if (b + 1 < kb) {
            la.load(A, K, m0, M, (b + 1) * FB_BK, K);
            lw.load(W, K, n0, N, (b + 1) * FB_BK, K);
        }
        i32x8 fa[2][2], fw[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                fa[t][ks] = frag32(&sA[buf][(arow + 32 * t) * FB_PITCH + 64 * ks + koff]);
                fw[t][ks] = frag32(&sW[buf][(wrow + 32 * t) * FB_PITCH + 64 * ks + koff]);
            }
        const float wsb = wsr[b];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            const float s = asr[ti][b] * wsb;
#pragma unroll
            for (int tj = 0; tj < 2; ++tj) {
                f32x16 p = {};
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[tj][ks], fa[ti][ks], p,
                                                                        0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[ti][tj][r] = __builtin_fmaf(p[r], s, acc[ti][tj][r]);
            }
        }
        if (b + 1 < kb) {
            la.store(sA[buf ^ 1]);
            lw.store(sW[buf ^ 1]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int ti = 0; ti < 2; ++ti)
#pragma unroll
        for (int tj = 0; tj < 2; ++tj)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t gj = n0 + wn * 64 + 32 * tj + mfma32_row(r, lane);
                if (row[ti] < M && gj < N)
                    out[(size_t)row[ti] * N + gj] = (uint16_t)f32_to_bf16(acc[ti][tj][r]);
            }
}

} // namespace

hipError_t launch_fp8_gemm_blockscale(const uint8_t *a, const float *as, const uint8_t *w,
                                      const float *ws, uint16_t *out, uint32_t m, uint32_t n,
                                      uint32_t k, hipStream_t st)
{
    const uint32_t mt = (m + FB_T - 1) / FB_T, nt = (n + FB_T - 1) / FB_T;
    hipLaunchKernelGGL(k_fp8_gemm_block, dim3(mt * nt), dim3(256), 0, st, a, as, w, ws, out, m, n, k,
                       mt, nt);
    count_launch();
    return hipGetLastError();
}

} // namespace qp
