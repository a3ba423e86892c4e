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
constexpr int kXPitch = kChunk * 2 + 64;  // bytes of a token's chunk: two tokens' reads meet
                                          // in different halves of the banks

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

template <int DT>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (DT == MOE_DT_BF16) asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma2_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// 8 codes (nibble i = value i) -> exact 16-bit pairs in the order x_pairs gives
// x: (0, 4), (1, 5), (2, 6), (3, 7), or (0, 1), ... for f16 E2M1.
// u4: a nibble in the low mantissa bits of 128 (bf16) or 1024 (f16) reads 128 + n
// or 1024 + n, and the zero point comes off with it, exactly (z: 128 + zero or
// 1024 + zero, twice).  f16 has room for the second nibble where it stands:
// 1024 + 16 n, times 1/16, minus 64 + zero (z2: its negative, twice).
// E2M1: f16 by the conversion instruction.  bf16: sign and magnitude bits placed at
// the sign and at the lowest exponent bits read the value times 2^-126 (0.5 as a
// subnormal); one multiplication brings it back, exactly.
template <int DT, int FMT>
__device__ __forceinline__ void expand(uint32_t v, uint32_t z, uint32_t z2, uint32_t (&o)[4]) {
  if constexpr (FMT == MOE_W4_U4 && DT == MOE_DT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = sub2<DT>(((v >> (4 * i)) & 0x000f000fu) | 0x43004300u, z);
  } else if constexpr (FMT == MOE_W4_U4) {
    const uint32_t u = v >> 8;
    o[0] = sub2<DT>((v & 0x000f000fu) | 0x64006400u, z);
    o[1] = fma2_f16((v & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, z2);
    o[2] = sub2<DT>((u & 0x000f000fu) | 0x64006400u, z);
    o[3] = fma2_f16((u & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, z2);
  } else if constexpr (DT == MOE_DT_F16) {
    e2m1x8_to_f16x2x4(v, o);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int up = 6 - 4 * i;  // nibble i's lowest bit goes to bit 6
      const uint32_t a = (up >= 0 ? v << (up >= 0 ? up : 0) : v >> (up >= 0 ? 0 : -up)) & 0x01c001c0u;
      o[i] = mul2_bf16(((v << (12 - 4 * i)) & 0x80008000u) | a, 0x7e807e80u);
    }
  }
}
template <int DT, int FMT>
__device__ __forceinline__ void x_pairs(const uint4& v, uint32_t (&o)[4]) {
  if constexpr (DT == MOE_DT_F16 && FMT == MOE_W4_E2M1) {
    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
  } else {
    o[0] = __byte_perm(v.x, v.z, 0x5410);
    o[1] = __byte_perm(v.x, v.z, 0x7632);
    o[2] = __byte_perm(v.y, v.w, 0x5410);
    o[3] = __byte_perm(v.y, v.w, 0x7632);
  }
}

// G32: the group's length in blocks of 32 values where it divides a chunk (1,
// 2 or 4: the group's end is known at compile time), 0: any
template <int DT, int FMT, int MT, int NT, int G32>
__global__ void __launch_bounds__(kMaxWarps * 32) k_w4(W4Args a) {
  constexpr int ROWS = 16 * MT;
  constexpr int STAGE = ROWS * kChunk / 2;  // bytes of one warp's stage of codes
  extern __shared__ __align__(128) uint8_t sm[];
  const int warps = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;
  const int n0 = blockIdx.x * ROWS, t0 = blockIdx.y * kTokens;
  const int nt = min(a.T - t0, NT * 8);  // tokens of this CTA
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int64_t krow = a.K / 2;
  const int xstage = nt * kXPitch;
  // all warps' rings of codes, then of x; then scale (high half) and zero point
  // of each row and group, rows an odd number of words apart
  const uint32_t cring = ptx::smem_u32(sm) + w * kStages * STAGE;
  uint8_t* xbase = sm + warps * kStages * STAGE + w * kStages * xstage;
  uint32_t* sz = (uint32_t*)(sm + warps * kStages * (STAGE + xstage));
  const int pitch = a.G | 1;
  pdl_wait();
  pdl_launch_dependents();

  auto issue = [&](int kc, int stage) {
    if (kc < chunks) {
      const int64_t at = (int64_t)kc * (kChunk / 2) + (lane & 7) * 16;
      const int r0 = lane >> 3;
      const uint8_t* src = a.codes + (n0 + r0) * krow + at;
      const bool in = at < krow;
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) {
        const int row = i * 4 + r0;
        const bool ok = in && n0 + row < a.N;
        cp_async16(cring + stage * STAGE + row * 128 + ((lane & 7) ^ (row & 7)) * 16,
                   ok ? src + i * 4 * krow : a.codes, ok ? 16 : 0);
      }
      const int k = kc * kChunk + lane * 8;
      const bool xin = k < a.K;
      const uint16_t* xs = a.x + t0 * a.ldx + (xin ? k : 0);
      uint32_t xd = ptx::smem_u32(xbase) + stage * xstage + lane * 16;
      for (int t = 0; t < nt; ++t, xs += a.ldx, xd += kXPitch) cp_async16(xd, xs, xin ? 16 : 0);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(w + i * warps, i);

  // (scales of the CTA's rows are one run of memory; loads of a batch leave together)
  const int entries = min(ROWS, a.N - n0) * a.G;
  for (int i0 = threadIdx.x; i0 < entries; i0 += 8 * blockDim.x) {
    uint32_t v[8], row[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * blockDim.x;
      row[k] = 0, v[k] = 0;
      if (i >= entries) continue;
      row[k] = i / a.G;
      v[k] = (uint32_t)a.scales[(int64_t)n0 * a.G + i] << 16;
      if constexpr (FMT == MOE_W4_U4) {
        const uint32_t grp = i - row[k] * a.G;
        v[k] |= a.zeros ? (a.zeros[(n0 + row[k]) * (int64_t)a.zrow + grp / 2] >> (4 * (grp & 1))) & 15
                        : 8;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * blockDim.x;
      if (i < entries) sz[row[k] * pitch + i - row[k] * a.G] = v[k];
    }
  }
  __syncthreads();

  float acc[MT][NT][4] = {}, sum[MT][NT][4] = {};
  int stage = 0;
  for (int kc = w; kc < chunks; kc += warps) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue(kc + (kStages - 1) * warps, stage == 0 ? kStages - 1 : stage - 1);
    const uint32_t cb = cring + stage * STAGE;
    const uint8_t* xb = xbase + stage * xstage + g * kXPitch + c4 * 16;
    const int blocks = min(8, a.K / 32 - kc * 8);  // of 32 values, in this chunk
    // the scale group, and what is left of it in blocks
    int grp = G32 ? kc * (8 / (G32 ? G32 : 1)) : kc * 8 / a.g32;
    int left = G32 ? 0 : (grp + 1) * a.g32 - kc * 8;
    uint32_t s[MT][2], z[MT][2], z2[MT][2];
    auto begin_group = [&]() {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s[m][r] = sz[(m * 16 + r * 8 + g) * pitch + grp];
          if constexpr (FMT == MOE_W4_U4) {
            const uint32_t zz = (s[m][r] & 0xffffu) * 0x00010001u;
            z[m][r] = (DT == MOE_DT_BF16 ? 0x43004300u : 0x64006400u) + zz;
            // -(64 + zero): 0x5400 is 64, whose last place is 1/16
            z2[m][r] = DT == MOE_DT_BF16 ? 0u : 0xd400d400u + zz * 16u;
          }
        }
    };
    begin_group();
    auto block = [&](int j, bool last) {
        uint32_t cw[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int row = m * 16 + (lane & 15);
          ldmatrix_x2(cw[m], cb + row * 128 + (j ^ (row & 7)) * 16);
        }
        uint32_t xp[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (n * 8 + g < nt) v = *(const uint4*)(xb + n * 8 * kXPitch + j * 64);
          x_pairs<DT, FMT>(v, xp[n]);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t p[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) expand<DT, FMT>(cw[m][r], z[m][r], z2[m][r], p[r]);
          const uint32_t lo[4] = {p[0][0], p[1][0], p[0][1], p[1][1]};
          const uint32_t hi[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816<DT>(sum[m][n], lo, xp[n][0], xp[n][1]);
            mma16816<DT>(sum[m][n], hi, xp[n][2], xp[n][3]);
          }
        }
        // the group ends here, or this warp's part of it does
        const bool end = G32 ? (j + 1) % (G32 ? G32 : 1) == 0 : --left == 0 || last;
        if (end) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float f = to_f32<DT>((uint16_t)(s[m][r] >> 16));
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  acc[m][n][2 * r + q] += f * sum[m][n][2 * r + q];
                  sum[m][n][2 * r + q] = 0.f;
                }
            }
          if (!last) {
            ++grp;
            if (!G32) left = a.g32;
            begin_group();
          }
        }
    };
    if (blocks == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) block(j, j == 7);
    } else {
#pragma unroll 1
      for (int j = 0; j < blocks; j += G32 ? G32 : 1)
#pragma unroll
        for (int k = 0; k < (G32 ? G32 : 1); ++k) block(j + k, j + k + 1 == blocks);
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
    const int ln = i & 31, q = (i >> 5) & 3, n = (i >> 7) % NT, m = (i >> 7) / NT;
    const int row = n0 + m * 16 + (q >> 1) * 8 + (ln >> 2);
    const int t = n * 8 + (ln & 3) * 2 + (q & 1);
    if (row < a.N && t < nt) {
      float v = 0.f;
      for (int k = 0; k < warps; ++k) v += red[k * MT * NT * 128 + i];
      if (a.bias) v += to_f32<DT>(a.bias[row]);
      a.y[(t0 + t) * a.ldy + row] = from_f32<DT>(v);
    }
  }
}

template <int DT, int FMT, int MT, int NT, int G32>
moe_status launch_w4(const W4Args& a, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return launch_status(cudaErrorUnknown);
  const uint64_t bit = 1ull << (dev & 63);
  constexpr size_t kMost = 227 * 1024;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        k_w4<DT, FMT, MT, NT, G32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return launch_status(e);
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int rows = 16 * MT, chunks = (a.K + kChunk - 1) / kChunk;
  const int nt = a.T < NT * 8 ? a.T : NT * 8;
  const size_t per_warp = (size_t)kStages * (rows * (kChunk / 2) + nt * kXPitch);
  const size_t table = (size_t)rows * (a.G | 1) * 4;
  int warps = chunks < kMaxWarps ? chunks : kMaxWarps;
  while (warps > 1 && warps * per_warp + table > kMost) --warps;
  const dim3 grid((a.N + rows - 1) / rows, (a.T + kTokens - 1) / kTokens);
  return launch_status(launch_pdl(k_w4<DT, FMT, MT, NT, G32>, grid, warps * 32,
                                  warps * per_warp + table, s, a));
}

template <int DT, int FMT, int MT, int NT>
moe_status pick_group(const W4Args& a, cudaStream_t s) {
  if (a.g32 == 1) return launch_w4<DT, FMT, MT, NT, 1>(a, s);
  if (a.g32 == 2) return launch_w4<DT, FMT, MT, NT, 2>(a, s);
  if (a.g32 == 4) return launch_w4<DT, FMT, MT, NT, 4>(a, s);
  return launch_w4<DT, FMT, MT, NT, 0>(a, s);
}

template <int DT, int FMT>
moe_status pick_w4(const W4Args& a, cudaStream_t s) {
  if (a.T <= 8) return pick_group<DT, FMT, 1, 1>(a, s);
  return pick_group<DT, FMT, 2, 2>(a, s);
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
