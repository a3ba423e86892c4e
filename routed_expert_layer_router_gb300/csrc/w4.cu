// w4.cu - K-w4: linear products of a few tokens with 4-bit weights that carry
// a scale (and zero point) per group of input values (moe_w4_linear).
//
// y[t][n] = sum_G s[n][G] * sum_{k in G} (value(code) - zero) x[t][k] + bias[n]
//
// Bound by reading the codes once: half a byte a weight, so the instructions per
// weight decide.  A warp takes 16 rows of W and every n-th chunk of 256 input
// values; it streams its codes through its own ring of cp.async stages.  ldmatrix
// on the raw codes hands a thread 8 consecutive codes of a row, four threads 32:
// that is one scale group of 32 or a part of a larger one, so every group size
// sums inside the matrix instructions in fp32 and the scale multiplies once a
// group.  Codes become exact 16-bit numbers by bit operations (the order of a
// product's terms is free: x takes the same order as the codes' nibbles).
// The warps that share a chunk (WR of them, for different rows) share its x in
// shared memory.  The K split of a CTA (WK) and of a cluster is added up in a
// fixed order at the end, the cluster's through distributed shared memory.
#include <atomic>

#include "elem.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int kChunk = 256;            // input values of a stage: 128 bytes of a row
constexpr int kTokens = 16;            // tokens of one pass over the weights
constexpr int kXPitch = kChunk * 2 + 64;  // bytes of a token's chunk: two tokens' reads meet
                                          // in different halves of the banks

struct W4Args {
  int T, N, K, G, g32, zrow;           // G groups of 32 * g32 values; zero bytes a row
  int wk;                              // warps along K in a CTA
  const uint16_t* x;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldx, ldy;
};

// The two 16-bit types of x, and how codes reach the matrix instructions.  Packed
// 16-bit arithmetic is slow on this GPU (four subtractions a word cost the
// kernel a third of its time), so no value is computed on its way: codes become
// operands by masks and shifts alone, and zero points ride along as operands.
//   u4, bf16: a nibble in the low mantissa bits of 128 reads 128 + n.
//   u4, f16: a nibble alone reads the subnormal n 2^-24; the second nibble of a
//     byte, where it stands, 16 n 2^-24 (summed apart and divided by 16).
//   Each instruction takes 8 input values twice, once with the codes and once with
//     -(128 + zero) or -zero, so the offset cancels before a sum is rounded.
//   E2M1: by the conversion instruction to f16.  A bf16 x goes to f16 in shared
//     memory under a power of two for each chunk of a token, which brings its
//     largest value to [2^14, 2^15): exact but for values 2^-29 below that.
template <int DT, int FMT>
struct Codes {
  static constexpr bool U4 = FMT == MOE_W4_U4;
  static constexpr bool TURN = DT == MOE_DT_BF16 && !U4;     // x: bf16 -> f16
  static constexpr int MT = TURN ? MOE_DT_F16 : DT;          // operands' type
  static constexpr int SETS = U4 && DT == MOE_DT_F16 ? 2 : 1;  // sums kept apart
  static constexpr float UNIT = SETS == 2 ? 16777216.f : 1.f;  // 2^24
};
// 8 codes (nibble i = value i) -> pairs (0, 4), (1, 5), (2, 6), (3, 7) for u4,
// (0, 1), (2, 3), ... for E2M1; x_pairs gives x in the same order
template <int DT, int FMT>
__device__ __forceinline__ void expand(uint32_t v, uint32_t (&o)[4]) {
  if constexpr (FMT == MOE_W4_E2M1) {
    e2m1x8_to_f16x2x4(v, o);
  } else if constexpr (DT == MOE_DT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = ((v >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  } else {
    const uint32_t u = v >> 8;
    o[0] = v & 0x000f000fu;
    o[1] = v & 0x00f000f0u;
    o[2] = u & 0x000f000fu;
    o[3] = u & 0x00f000f0u;
  }
}
template <int FMT>
__device__ __forceinline__ void x_pairs(const uint4& v, uint32_t (&o)[4]) {
  if constexpr (FMT == MOE_W4_E2M1) {
    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
  } else {
    o[0] = __byte_perm(v.x, v.z, 0x5410);
    o[1] = __byte_perm(v.x, v.z, 0x7632);
    o[2] = __byte_perm(v.y, v.w, 0x5410);
    o[3] = __byte_perm(v.y, v.w, 0x7632);
  }
}
// 8 bf16 values a lane (a token's chunk a warp) -> f16 under one power of two;
// returns what undoes it
__device__ __forceinline__ float turn_to_f16(uint4& v) {
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                        __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  m = __reduce_max_sync(~0u, max(m & 0xffffu, m >> 16));
  // exponent of the largest value; infinities and NaN keep their meaning under
  // any power, the finite values beside them come down with 2^127
  const int e = min((int)(m >> 7), 254) - 127;
  const int up = m == 0 ? 0 : min(14 - e, 100);
  const float f = __uint_as_float((uint32_t)(127 + up) << 23);
  v.x = pack_f16(bf16_lo(v.x) * f, bf16_hi(v.x) * f);
  v.y = pack_f16(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
  v.z = pack_f16(bf16_lo(v.z) * f, bf16_hi(v.z) * f);
  v.w = pack_f16(bf16_lo(v.w) * f, bf16_hi(v.w) * f);
  return __uint_as_float((uint32_t)(127 - up) << 23);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// fp32 at the address of this CTA's shared memory, read from CTA `rank` of the cluster
__device__ __forceinline__ float cluster_load(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n"
               " ld.shared::cluster.f32 %0, [a];\n}"
               : "=f"(v)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}

// WR: warps along the rows of W, which share x.  G32: the group's length in
// blocks of 32 values where it divides a chunk (1, 2, 4), 8 where chunks divide
// it, 0 for any other: the scales of the next chunk are then not fetched ahead.
template <int DT, int FMT, int NT, int WR, int G32>
__global__ void __launch_bounds__(256) k_w4(W4Args a) {
  using C = Codes<DT, FMT>;
  constexpr int S = WR == 1 ? 4 : 3;        // stages
  constexpr int STAGE = 16 * kChunk / 2;    // bytes of one warp's stage of codes
  constexpr int NG = G32 ? 8 / G32 : 1;     // groups of a chunk
  constexpr int SV = NG == 8 ? 2 : 1;       // of which a lane fetches this many
  extern __shared__ __align__(128) uint8_t sm[];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = w % WR, kw = w / WR;       // place along rows, along K
  const int g = lane >> 2, c4 = lane & 3;
  const int crank = cluster_rank(), csize = cluster_size();
  const int n0 = (blockIdx.x / csize) * 16 * WR + wr * 16, t0 = blockIdx.y * kTokens;
  const int nt = min(a.T - t0, NT * 8);     // tokens of this CTA
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int step = a.wk * csize;            // this warp: chunks first, first + step, ...
  const int first = crank * a.wk + kw;
  const int64_t krow = a.K / 2;
  const int xstage = nt * kXPitch;
  __shared__ float undo[8 / WR][kTokens];   // E2M1, bf16: of each chunk in work
  const uint32_t cring = ptx::smem_u32(sm) + w * S * STAGE;
  uint8_t* xbase = sm + a.wk * WR * S * STAGE + kw * S * xstage;
  pdl_wait();
  pdl_launch_dependents();

  // per lane: rows r0, r0 + 4, ... of the codes; per group of WR warps: x
  const int r0 = lane >> 3;
  const uint8_t* csrc = a.codes + (n0 + r0) * krow + (lane & 7) * 16;
  const uint32_t cdst = cring + r0 * 128;
  uint32_t on = 0;  // bit i: row i * 4 + r0 exists
#pragma unroll
  for (int i = 0; i < 4; ++i) on |= (n0 + i * 4 + r0 < a.N ? 1u : 0u) << i;
  auto issue = [&](int kc, int stage) {
    if (kc < chunks) {
      const bool in = kc * (kChunk / 2) + (lane & 7) * 16 < krow;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = in && ((on >> i) & 1);
        cp_async16(cdst + stage * STAGE + i * 512 + (((lane & 7) ^ (i * 4 + r0)) & 7) * 16,
                   ok ? csrc + i * 4 * krow + kc * (kChunk / 2) : a.codes, ok ? 16 : 0);
      }
      const int k = kc * kChunk + lane * 8;
      const bool xin = k < a.K;
      const uint16_t* xs = a.x + (t0 + wr) * a.ldx + (xin ? k : 0);
      uint32_t xd = ptx::smem_u32(xbase) + stage * xstage + wr * kXPitch + lane * 16;
      for (int t = wr; t < nt; t += WR, xs += WR * a.ldx, xd += WR * kXPitch)
        cp_async16(xd, xs, xin ? 16 : 0);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(first + i * step, i);

  // scale (high half) and zero point of row r * 8 + g and group grp
  auto scale_word = [&](int r, int grp) {
    const int row = n0 + r * 8 + g;
    uint32_t v = 0;
    if (row < a.N && grp < a.G) {
      v = (uint32_t)a.scales[(int64_t)row * a.G + grp] << 16;
      if constexpr (FMT == MOE_W4_U4)
        v |= a.zeros ? (a.zeros[(int64_t)row * a.zrow + grp / 2] >> (4 * (grp & 1))) & 15 : 8;
    }
    return v;
  };
  // the four lanes of a row fetch one group each (two each of eight)
  uint32_t cur[2][SV] = {}, nxt[2][SV] = {};
  auto fetch_scales = [&](int kc) {
    if constexpr (G32 != 0) {
      if (kc >= chunks) return;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int v = 0; v < SV; ++v)
          nxt[r][v] = scale_word(r, G32 == 8 ? kc * 8 / a.g32 : kc * NG + v * 4 + c4 % NG);
    }
  };
  fetch_scales(first);

  float acc[NT][4] = {}, sum[C::SETS][NT][4] = {};
  int stage = 0;
  auto group_sync = [&]() {  // the warps that share a chunk
    if constexpr (WR == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + kw), "n"(WR * 32) : "memory");
  };
  for (int kc = first; kc < chunks; kc += step) {
    cp_async_wait<S - 2>();
    group_sync();
    issue(kc + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int v = 0; v < SV; ++v) cur[r][v] = nxt[r][v];
    fetch_scales(kc + step);
    const uint32_t cb = cring + stage * STAGE + (lane & 15) * 128;
    const uint8_t* xb = xbase + stage * xstage + g * kXPitch + c4 * 16;
    const int blocks = min(8, a.K / 32 - kc * 8);  // of 32 values, in this chunk
    float back[NT][2];
    if constexpr (C::TURN) {
      for (int t = wr; t < nt; t += WR) {
        uint4* p = (uint4*)(xbase + stage * xstage + t * kXPitch + lane * 16);
        uint4 v = *p;
        const float u = turn_to_f16(v);
        *p = v;
        if (lane == 0) undo[kw][t] = u;
      }
      group_sync();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) back[n][q] = undo[kw][n * 8 + c4 * 2 + q];
    }
    // G32 == 0: the scale group, and what is left of it in blocks
    int grp = G32 ? 0 : kc * 8 / a.g32;
    int left = G32 ? 0 : (grp + 1) * a.g32 - kc * 8;
    uint32_t s[2], z[2];
    auto begin_group = [&](int local) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (G32 == 0) s[r] = scale_word(r, grp);
        else if (NG == 1) s[r] = cur[r][0];
        else s[r] = __shfl_sync(~0u, cur[r][local / 4 % SV], (lane & 28) | (local & 3));
        if constexpr (C::U4)  // -(128 + zero), or -zero as a subnormal, twice
          z[r] = (s[r] & 0xffffu) * 0x00010001u | (DT == MOE_DT_BF16 ? 0xc300c300u : 0x80008000u);
      }
    };
    begin_group(0);
    auto block = [&](int j, bool last) {
      uint32_t cw[2];
      ldmatrix_x2(cw, cb + ((j ^ lane) & 7) * 16);
      uint32_t xp[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (n * 8 + g < nt) v = *(const uint4*)(xb + n * 8 * kXPitch + j * 64);
        x_pairs<FMT>(v, xp[n]);
      }
      uint32_t p[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) expand<DT, FMT>(cw[r], p[r]);
      if constexpr (C::U4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          constexpr bool two = C::SETS == 2;
          const uint32_t f[4] = {p[0][i], p[1][i], two && (i & 1) ? (z[0] & 0x000f000fu) << 4 | 0x80008000u : z[0],
                                 two && (i & 1) ? (z[1] & 0x000f000fu) << 4 | 0x80008000u : z[1]};
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<C::MT>(sum[two ? i & 1 : 0][n], f, xp[n][i], xp[n][i]);
        }
      } else {
        const uint32_t lo[4] = {p[0][0], p[1][0], p[0][1], p[1][1]};
        const uint32_t hi[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816<C::MT>(sum[0][n], lo, xp[n][0], xp[n][1]);
          mma16816<C::MT>(sum[0][n], hi, xp[n][2], xp[n][3]);
        }
      }
      // the group ends here, or this warp's part of it does
      const bool end = G32 ? (j + 1) % (G32 ? G32 : 1) == 0 || last : --left == 0 || last;
      if (end) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = to_f32<DT>((uint16_t)(s[r] >> 16)) * C::UNIT;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int k = 2 * r + q;
              float v = sum[0][n][k];
              sum[0][n][k] = 0.f;
              if constexpr (C::SETS == 2) {
                v += sum[1][n][k] * 0.0625f;
                sum[1][n][k] = 0.f;
              }
              if constexpr (C::TURN) v *= back[n][q];
              acc[n][k] += f * v;
            }
        }
        if (!last) {
          if (!G32) ++grp, left = a.g32;
          begin_group(G32 ? (j + 1) / (G32 ? G32 : 1) : 0);
        }
      }
    };
    if (blocks == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) block(j, j == 7);
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < blocks) block(j, j + 1 == blocks);
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  __syncthreads();

  // sums over the warps along K in their order, then over the cluster in rank
  // order; the outputs are dealt to its CTAs
  constexpr int OUT = WR * NT * 128;
  float* red = (float*)sm;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[(w * NT + n) * 128 + q * 32 + lane] = acc[n][q];
  __syncthreads();
  if (csize > 1) {
    for (int i = threadIdx.x; i < OUT; i += blockDim.x) {
      float v = red[i];
      for (int k = 1; k < a.wk; ++k) v += red[k * OUT + i];
      red[i] = v;
    }
    cluster_sync();
  }
  const uint32_t red_addr = ptx::smem_u32(red);
  for (int i = threadIdx.x + crank * blockDim.x; i < OUT; i += blockDim.x * csize) {
    const int ln = i & 31, q = (i >> 5) & 3, n = (i >> 7) % NT, m = (i >> 7) / NT;
    const int row = (blockIdx.x / csize) * 16 * WR + m * 16 + (q >> 1) * 8 + (ln >> 2);
    const int t = n * 8 + (ln & 3) * 2 + (q & 1);
    if (row < a.N && t < nt) {
      float v = 0.f;
      if (csize > 1) {
        for (int k = 0; k < csize; ++k) v += cluster_load(red_addr + i * 4, k);
      } else {
        for (int k = 0; k < a.wk; ++k) v += red[k * OUT + i];
      }
      if (a.bias) v += to_f32<DT>(a.bias[row]);
      a.y[(t0 + t) * a.ldy + row] = from_f32<DT>(v);
    }
  }
  if (csize > 1) cluster_sync();  // until all have read
}

template <int DT, int FMT, int NT, int WR, int G32>
moe_status launch_w4(W4Args a, cudaStream_t s) {
  auto* kern = k_w4<DT, FMT, NT, WR, G32>;
  constexpr int S = WR == 1 ? 4 : 3;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return launch_status(cudaErrorUnknown);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return launch_status(e);
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int tiles = (a.N + 16 * WR - 1) / (16 * WR), passes = (a.T + kTokens - 1) / kTokens;
  const int nt = a.T < NT * 8 ? a.T : NT * 8;
  // warps along K: 8 in all, but 4 where the rows alone bring 12 warps an SM
  // (longer runs of chunks a warp, fewer beginnings); then a cluster along K while
  // SMs are left without a CTA
  a.wk = 8 / WR;
  if (WR == 1 && (int64_t)tiles * passes * 4 >= 8 * kSMs) a.wk = 4;
  if (a.wk > chunks) a.wk = chunks;
  int cluster = 1;
  while (cluster < 8 && (int64_t)tiles * passes * cluster < (WR == 1 ? kSMs / 2 : kSMs + kSMs / 4) &&
         a.wk * cluster * 2 <= chunks)
    cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * cluster, passes);
  cfg.blockDim = dim3(a.wk * WR * 32);
  cfg.dynamicSmemBytes = (size_t)a.wk * S * (WR * 16 * (kChunk / 2) + nt * kXPitch);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return launch_status(cudaLaunchKernelEx(&cfg, kern, a));
}

template <int DT, int FMT, int NT, int WR>
moe_status pick_group(const W4Args& a, cudaStream_t s) {
  if (a.g32 == 1) return launch_w4<DT, FMT, NT, WR, 1>(a, s);
  if (a.g32 == 2) return launch_w4<DT, FMT, NT, WR, 2>(a, s);
  if (a.g32 == 4) return launch_w4<DT, FMT, NT, WR, 4>(a, s);
  if (a.g32 % 8 == 0) return launch_w4<DT, FMT, NT, WR, 8>(a, s);
  return launch_w4<DT, FMT, NT, WR, 0>(a, s);
}

template <int DT, int FMT>
moe_status pick_w4(const W4Args& a, cudaStream_t s) {
  if (a.T <= 2) return pick_group<DT, FMT, 1, 1>(a, s);
  if (a.T <= 8) return pick_group<DT, FMT, 1, 4>(a, s);
  return pick_group<DT, FMT, 2, 4>(a, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_w4_linear(const moe_w4_linear_args* a, void* stream) {
  if (!a || a->T < 0 || a->N <= 0 || a->K <= 0 || a->group <= 0) return MOE_ERR_INVALID_ARG;
  if (a->format != MOE_W4_U4 && a->format != MOE_W4_E2M1) return MOE_ERR_INVALID_ARG;
  if (a->format == MOE_W4_E2M1 && a->zeros) return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
  if (a->group % 32 || a->K % a->group) return MOE_ERR_UNSUPPORTED;
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
