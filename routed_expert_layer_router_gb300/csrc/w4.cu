// w4.cu - K-w4: linear products of a few tokens with 4-bit weights that carry
// a scale (and zero point) per group of input values (moe_w4_linear).
//
// y[t][n] = sum_G s[n][G] * sum_{k in G} (value(code) - zero) x[t][k] + bias[n]
//
// Bound by reading the codes once: half a byte a weight, so the work per weight
// has to stay near one instruction a thread for two weights.  A CTA takes
// 16 * MT rows of W; its warps take every WARPS-th chunk of 256 input values.
// Each warp streams its chunks through its own ring of cp.async stages and
// needs no barrier until the end, where the warps' sums are added in warp
// order.  ldmatrix on the raw codes hands a thread 8 consecutive codes of a row,
// four threads 32: that is one scale group of 32 or a part of a larger one, so
// every group size sums inside the matrix instructions in fp32 and the scale
// multiplies once a group.  Codes become exact 16-bit numbers by bit operations
// (the order of a product's terms is free: x takes the same order as the codes'
// nibbles).  x comes straight from L1 / L2 in 16-byte loads.
#include <atomic>

#include "elem.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int kChunk = 256;            // input values of a stage: 128 bytes of a row
constexpr int kMaxWarps = 8;
constexpr int kStages = 4;
constexpr int kTokens = 16;            // tokens of one pass over the weights

struct W4Args {
  int T, N, K, G, g32, zrow;           // G groups of 32 * g32 values; zero bytes a row
  const uint16_t* x;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldx, ldy;
};

__device__ __forceinline__ uint32_t sub2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t sub2_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul2_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 8 codes (nibble i = value i) -> pairs (0, 4), (1, 5), (2, 6), (3, 7).
// u4: a nibble placed in the mantissa of 128 (bf16) or 1024 (f16) gives 128 + n
// or 1024 + n; `zc` (128 or 1024 plus the zero point, twice) comes off exactly.
// E2M1: sign and the three magnitude bits placed at the sign and at the lowest
// exponent bits give the value times 2^-126 or 2^-14 (0.5 as a subnormal); one
// multiplication brings it back, exactly.
template <int DT, int FMT>
__device__ __forceinline__ void expand(uint32_t v, uint32_t zc, uint32_t (&o)[4]) {
  if constexpr (FMT == MOE_W4_U4) {
    constexpr uint32_t one = DT == MOE_DT_BF16 ? 0x43004300u : 0x64006400u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t n = ((v >> (4 * i)) & 0x000f000fu) | one;
      o[i] = DT == MOE_DT_BF16 ? sub2_bf16(n, zc) : sub2_f16(n, zc);
    }
  } else {
    constexpr int top = DT == MOE_DT_BF16 ? 8 : 11;  // bit of the magnitude's top bit
    constexpr uint32_t mag = 7u << (top - 2), mask = mag | mag << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int up = top - 2 - 4 * i;  // where nibble i's lowest bit has to go
      const uint32_t a = (up >= 0 ? v << (up >= 0 ? up : 0) : v >> (up >= 0 ? 0 : -up)) & mask;
      const uint32_t n = ((v << (12 - 4 * i)) & 0x80008000u) | a;
      o[i] = DT == MOE_DT_BF16 ? mul2_bf16(n, 0x7e807e80u) : mul2_f16(n, 0x74007400u);
    }
  }
}

template <int DT, int FMT, int MT, int NT>
__global__ void __launch_bounds__(kMaxWarps * 32) k_w4(W4Args a) {
  constexpr int ROWS = 16 * MT;
  constexpr int STAGE = ROWS * kChunk / 2;  // bytes of one warp's stage
  extern __shared__ __align__(128) uint8_t sm[];
  const int warps = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;
  uint8_t* ring = sm + w * kStages * STAGE;
  // scales (row stride odd in 4-byte words: no bank conflicts over rows) and zeros
  const int srow = (a.G + 1) / 2 * 2 + ((a.G + 1) / 2 % 2 ? 0 : 2);
  uint16_t* ssc = (uint16_t*)(sm + warps * kStages * STAGE);
  uint8_t* szr = (uint8_t*)(ssc + ROWS * srow);
  const int n0 = blockIdx.x * ROWS, t0 = blockIdx.y * kTokens;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int64_t krow = a.K / 2;
  pdl_wait();
  pdl_launch_dependents();

  const uint32_t rbase = ptx::smem_u32(ring);
  auto issue = [&](int kc, int stage) {
    if (kc < chunks) {
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) {
        const int row = i * 4 + (lane >> 3), ch = lane & 7;
        const int64_t at = (int64_t)kc * (kChunk / 2) + ch * 16;
        const bool ok = n0 + row < a.N && at < krow;
        cp_async16(rbase + stage * STAGE + row * 128 + (ch ^ (row & 7)) * 16,
                   a.codes + (ok ? (n0 + row) * krow + at : 0), ok ? 16 : 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(w + i * warps, i);

  const int rows = min(ROWS, a.N - n0);
  for (int i = threadIdx.x; i < rows * a.G; i += blockDim.x)
    ssc[(i / a.G) * srow + i % a.G] = a.scales[(int64_t)n0 * a.G + i];
  if (FMT == MOE_W4_U4 && a.zeros)
    for (int i = threadIdx.x; i < rows * a.zrow; i += blockDim.x)
      szr[i] = a.zeros[(int64_t)n0 * a.zrow + i];
  __syncthreads();

  // 128 or 1024 plus the zero point, twice, for this lane's rows
  auto load_zero = [&](int grp, uint32_t (&zc)[MT][2]) {
    if constexpr (FMT == MOE_W4_U4) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t z = 8;
          if (a.zeros && grp < a.G)
            z = (szr[(m * 16 + r * 8 + g) * a.zrow + grp / 2] >> (4 * (grp & 1))) & 15;
          zc[m][r] = (DT == MOE_DT_BF16 ? 0x43004300u : 0x64006400u) + (z | z << 16);
        }
    }
  };

  float acc[MT][NT][4] = {}, sum[MT][NT][4] = {};
  int stage = 0;
  for (int kc = w; kc < chunks; kc += warps) {
    // x of this chunk: lane (g, c4) holds 8 consecutive values of token g per 32
    uint4 xv[8][NT];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = t0 + n * 8 + g, k = kc * kChunk + j * 32 + c4 * 8;
        xv[j][n] = make_uint4(0, 0, 0, 0);
        if (t < a.T && k < a.K) xv[j][n] = *(const uint4*)(a.x + t * a.ldx + k);
      }
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue(kc + (kStages - 1) * warps, stage == 0 ? kStages - 1 : stage - 1);
    const uint32_t sb = rbase + stage * STAGE;
    // the scale group of the chunk's first block of 32 values, and the blocks
    // that are left in the group and in the row
    int grp = kc * 8 / a.g32, left = (grp + 1) * a.g32 - kc * 8;
    const int blocks = min(8, a.K / 32 - kc * 8);
    uint32_t zc[MT][2] = {};
    load_zero(grp, zc);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t cw[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + (lane & 15), ch = j + (lane >> 4);
        ldmatrix_x4(cw[m], sb + row * 128 + (ch ^ (row & 7)) * 16);
      }
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        uint32_t xp[NT][4];  // pairs (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = xv[j + jj][n];
          xp[n][0] = __byte_perm(v.x, v.z, 0x5410);
          xp[n][1] = __byte_perm(v.x, v.z, 0x7632);
          xp[n][2] = __byte_perm(v.y, v.w, 0x5410);
          xp[n][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t p[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r)
            expand<DT, FMT>(cw[m][2 * jj + r], zc[m][r], p[r]);
          const uint32_t lo[4] = {p[0][0], p[1][0], p[0][1], p[1][1]};
          const uint32_t hi[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816<DT>(sum[m][n], lo, xp[n][0], xp[n][1]);
            mma16816<DT>(sum[m][n], hi, xp[n][2], xp[n][3]);
          }
        }
        // the group ends here, or this warp's part of it does
        const int blk = j + jj;
        if (--left == 0 || blk == 7) {
          if (blk < blocks) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float s = to_f32<DT>(ssc[(m * 16 + r * 8 + g) * srow + grp]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int q = 0; q < 2; ++q) {
                    acc[m][n][2 * r + q] += s * sum[m][n][2 * r + q];
                    sum[m][n][2 * r + q] = 0.f;
                  }
              }
          }
          left = a.g32;
          ++grp;
          if (blk < 7) load_zero(grp, zc);
        }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  __syncthreads();

  // the warps' sums, added in warp order
  float* red = (float*)sm;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[((w * MT + m) * NT + n) * 128 + q * 32 + lane] = acc[m][n][q];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NT * 128; i += blockDim.x) {
    float v = 0.f;
    for (int k = 0; k < warps; ++k) v += red[k * MT * NT * 128 + i];
    const int ln = i & 31, q = (i >> 5) & 3, n = (i >> 7) % NT, m = (i >> 7) / NT;
    const int row = n0 + m * 16 + (q >> 1) * 8 + (ln >> 2);
    const int t = t0 + n * 8 + (ln & 3) * 2 + (q & 1);
    if (row < a.N && t < a.T) {
      if (a.bias) v += to_f32<DT>(a.bias[row]);
      a.y[t * a.ldy + row] = from_f32<DT>(v);
    }
  }
}

template <int DT, int FMT, int MT, int NT>
moe_status launch_w4(const W4Args& a, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return launch_status(cudaErrorUnknown);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        k_w4<DT, FMT, MT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return launch_status(e);
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int rows = 16 * MT, chunks = (a.K + kChunk - 1) / kChunk;
  const int warps = chunks < kMaxWarps ? chunks : kMaxWarps;
  const int srow = (a.G + 1) / 2 * 2 + ((a.G + 1) / 2 % 2 ? 0 : 2);
  const size_t ring = (size_t)warps * kStages * rows * (kChunk / 2);  // also the warps' sums
  const size_t smem = ring + (size_t)rows * (srow * 2 + a.zrow);
  const dim3 grid((a.N + rows - 1) / rows, (a.T + kTokens - 1) / kTokens);
  return launch_status(launch_pdl(k_w4<DT, FMT, MT, NT>, grid, warps * 32, smem, s, a));
}

template <int DT, int FMT>
moe_status pick_w4(const W4Args& a, cudaStream_t s) {
  if (a.T <= 8) return launch_w4<DT, FMT, 1, 1>(a, s);
  return launch_w4<DT, FMT, 2, 2>(a, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_w4_linear(const moe_w4_linear_args* a, void* stream) {
  if (!a || a->T < 0 || a->N <= 0 || a->K <= 0 || a->group <= 0) return MOE_ERR_INVALID_ARG;
  if (a->format != MOE_W4_U4 && a->format != MOE_W4_E2M1) return MOE_ERR_INVALID_ARG;
  if (a->format == MOE_W4_E2M1 && a->zeros) return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
  if (a->group % 32 || a->K % a->group || a->K / a->group > 1024) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  if (!a->x || !a->codes || !a->scales || !a->y || a->ldx < a->K || a->ldy < a->N)
    return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)a->x & 15) || ((uintptr_t)a->codes & 15) || a->ldx % 8)
    return MOE_ERR_UNSUPPORTED;
  if (a->T > kTokens * 65535) return MOE_ERR_UNSUPPORTED;
  W4Args k;
  k.T = a->T, k.N = a->N, k.K = a->K, k.G = a->K / a->group, k.g32 = a->group / 32;
  k.zrow = a->zeros ? (k.G + 1) / 2 : 0;
  k.x = (const uint16_t*)a->x, k.codes = a->codes, k.scales = (const uint16_t*)a->scales;
  k.zeros = a->zeros, k.bias = (const uint16_t*)a->bias, k.y = (uint16_t*)a->y;
  k.ldx = a->ldx, k.ldy = a->ldy;
  cudaStream_t s = (cudaStream_t)stream;
  if (a->dtype == MOE_DT_BF16)
    return a->format == MOE_W4_U4 ? pick_w4<MOE_DT_BF16, MOE_W4_U4>(k, s)
                                  : pick_w4<MOE_DT_BF16, MOE_W4_E2M1>(k, s);
  return a->format == MOE_W4_U4 ? pick_w4<MOE_DT_F16, MOE_W4_U4>(k, s)
                                : pick_w4<MOE_DT_F16, MOE_W4_E2M1>(k, s);
}
