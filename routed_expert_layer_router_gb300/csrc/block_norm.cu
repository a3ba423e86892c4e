// block_norm.cu - K-block-norm: the residual addition between two blocks with
// the norms on both sides of it, the block's gate and the residual scale, in
// one pass (formulas in moe.h).
//
// Bound by memory: x and y are read once, r and h written once.  A CTA owns a
// row and keeps it in registers as fp32 (kVec * VPT values a thread), so the
// statistics cost no second read; a layer norm's variance is taken around the
// mean from the registers.  Weights and channel gates come through L1 / L2.
#include "elem.cuh"

namespace moe {
namespace {

struct NormArgs {
  int T, H, kind, gate_act, post_norm, w16;
  const void *x, *y, *gate, *w_post, *b_post, *w_pre, *b_pre;
  void *r, *h;
  int64_t ldx, ldy, ldr, ldh, gate_row, gate_col;
  float res_scale, branch_scale, eps, w_offset;
};

template <int DT, int VEC>
__device__ __forceinline__ void load(const void* p, int64_t i, float (&v)[VEC]) {
  const typename Elem<DT>::T* q = (const typename Elem<DT>::T*)p + i;
  if constexpr (VEC == 1) v[0] = to_f32<DT>(*q);
  else load8<DT>(q, v);
}
template <int DT, int VEC>
__device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[VEC]) {
  typename Elem<DT>::T* q = (typename Elem<DT>::T*)p + i;
  if constexpr (VEC == 1) *q = from_f32<DT>(v[0]);
  else store8<DT>(q, v);
}

// sum over the CTA, the same bits in every thread; `slot` alternates between
// the two halves of `part` so that one barrier a sum is enough
__device__ __forceinline__ float block_sum(float v, float (*part)[32], int& slot) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_sum(lane < warps ? part[slot][lane] : 0.f);
  slot ^= 1;
  return v;
}

template <int RT, int BT, int VEC, int VPT>
__global__ void __launch_bounds__(1024) k_block_norm(NormArgs a) {
  __shared__ float part[2][32];
  int slot = 0;
  const int H = a.H, step = blockDim.x * VEC;
  const int i0 = threadIdx.x * VEC;
  const float inv_h = 1.f / (float)H;
  pdl_wait();
  pdl_launch_dependents();

  // v <- N(v; w, c), rows' statistics over the CTA
  auto norm = [&](float (&v)[VPT][VEC], const void* w, const void* c) {
    float mean = 0.f;
    if (a.kind == MOE_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (i0 + k * step < H)
#pragma unroll
          for (int j = 0; j < VEC; ++j) s += v[k][j];
      mean = block_sum(s, part, slot) * inv_h;
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (i0 + k * step < H)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[k][j] -= mean;
          s += v[k][j] * v[k][j];
        }
    const float rs = rsqrtf(block_sum(s, part, slot) * inv_h + a.eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = i0 + k * step;
      if (i < H) {
        float u[VEC];
        if (w) {
          if (a.w16) load<BT, VEC>(w, i, u);
          else load<MOE_DT_F32, VEC>(w, i, u);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[k][j] *= rs * (u[j] + a.w_offset);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[k][j] *= rs;
        }
        if (c) {
          if (a.w16) load<BT, VEC>(c, i, u);
          else load<MOE_DT_F32, VEC>(c, i, u);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[k][j] += u[j];
        }
      }
    }
  };

  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float r[VPT][VEC], b[VPT][VEC];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = i0 + k * step;
      if (i < H) {
        load<RT, VEC>(a.x, t * a.ldx + i, r[k]);
        if (a.y) load<BT, VEC>(a.y, t * a.ldy + i, b[k]);
      }
    }
    if (a.y) {
      if (a.post_norm) norm(b, a.w_post, a.b_post);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = i0 + k * step;
        if (i < H) {
          float g[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) g[j] = 1.f;
          if (a.gate) {
            if (a.gate_col) {
              load<BT, VEC>(a.gate, t * a.gate_row + i, g);
            } else {
              float one[1];
              load<BT, 1>(a.gate, t * a.gate_row, one);
#pragma unroll
              for (int j = 0; j < VEC; ++j) g[j] = one[0];
            }
            if (a.gate_act == MOE_GATE_SIGMOID)
#pragma unroll
              for (int j = 0; j < VEC; ++j) g[j] = 1.f / (1.f + expf(-g[j]));
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            r[k][j] = a.res_scale * r[k][j] + a.branch_scale * (g[j] * b[k][j]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) r[k][j] *= a.res_scale;
    }
    if (a.r) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = i0 + k * step;
        if (i < H) store<RT, VEC>(a.r, t * a.ldr + i, r[k]);
      }
    }
    if (a.h) {
      norm(r, a.w_pre, a.b_pre);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = i0 + k * step;
        if (i < H) store<BT, VEC>(a.h, t * a.ldh + i, r[k]);
      }
    }
  }
}

template <int RT, int BT, int VEC, int VPT>
cudaError_t launch(const NormArgs& a, int threads, cudaStream_t s) {
  return launch_pdl(k_block_norm<RT, BT, VEC, VPT>, a.T, threads, 0, s, a);
}

template <int RT, int BT>
cudaError_t dispatch(const NormArgs& a, bool vec, cudaStream_t s) {
  const int per = vec ? 8 : 1, units = (a.H + per - 1) / per;
  auto threads = [&](int vpt) { return ((units + vpt - 1) / vpt + 31) / 32 * 32; };
  if (vec) {
    if (threads(1) <= 1024) return launch<RT, BT, 8, 1>(a, threads(1), s);
    if (threads(2) <= 1024) return launch<RT, BT, 8, 2>(a, threads(2), s);
    return launch<RT, BT, 8, 4>(a, threads(4), s);
  }
  if (threads(4) <= 1024) return launch<RT, BT, 1, 4>(a, threads(4), s);
  return launch<RT, BT, 1, 32>(a, threads(32), s);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_block_norm(const moe_block_norm_args* a, void* stream) {
  if (!a || a->T < 0 || a->H <= 0) return MOE_ERR_INVALID_ARG;
  if (a->kind != MOE_NORM_RMS && a->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (a->gate_act != MOE_GATE_NONE && a->gate_act != MOE_GATE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (a->gate && ((a->gate_col != 0 && a->gate_col != 1) || a->gate_row < 0))
    return MOE_ERR_INVALID_ARG;
  const int RT = a->stream_type, BT = a->branch_type;
  const bool types = (RT == BT && (BT == MOE_DT_BF16 || BT == MOE_DT_F16 || BT == MOE_DT_F32)) ||
                     (RT == MOE_DT_F32 && (BT == MOE_DT_BF16 || BT == MOE_DT_F16));
  if (!types || (a->weight_type != MOE_DT_F32 && a->weight_type != BT)) return MOE_ERR_UNSUPPORTED;
  if (a->H > 32768) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  if (!a->r && !a->h) return MOE_ERR_INVALID_ARG;
  if (!a->y && (a->gate || a->post_norm)) return MOE_ERR_INVALID_ARG;
  if (!a->x || a->ldx < a->H || (a->y && a->ldy < a->H) || (a->r && a->ldr < a->H) ||
      (a->h && a->ldh < a->H))
    return MOE_ERR_INVALID_ARG;

  NormArgs k;
  k.T = a->T, k.H = a->H, k.kind = a->kind, k.gate_act = a->gate_act;
  k.post_norm = a->post_norm != 0, k.w16 = a->weight_type != MOE_DT_F32;
  k.x = a->x, k.y = a->y, k.gate = a->gate;
  k.w_post = a->w_post, k.b_post = a->b_post, k.w_pre = a->w_pre, k.b_pre = a->b_pre;
  k.r = a->r, k.h = a->h;
  k.ldx = a->ldx, k.ldy = a->ldy, k.ldr = a->ldr, k.ldh = a->ldh;
  k.gate_row = a->gate_row, k.gate_col = a->gate_col;
  k.res_scale = a->res_scale, k.branch_scale = a->branch_scale;
  k.eps = a->eps, k.w_offset = a->w_offset;

  // 16-byte accesses of 8 values where every row that is read or written
  // allows them; value by value otherwise
  auto aligned = [](const void* p, int64_t ld) {
    return !p || (((uintptr_t)p & 15) == 0 && ld % 8 == 0);
  };
  const bool vec = a->H % 8 == 0 && aligned(a->x, a->ldx) && aligned(a->y, a->ldy) &&
                   aligned(a->r, a->ldr) && aligned(a->h, a->ldh) && aligned(a->w_post, 0) &&
                   aligned(a->b_post, 0) && aligned(a->w_pre, 0) && aligned(a->b_pre, 0) &&
                   (!a->gate || a->gate_col == 0 || aligned(a->gate, a->gate_row));
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (RT == MOE_DT_BF16) e = dispatch<MOE_DT_BF16, MOE_DT_BF16>(k, vec, s);
  else if (RT == MOE_DT_F16) e = dispatch<MOE_DT_F16, MOE_DT_F16>(k, vec, s);
  else if (BT == MOE_DT_F32) e = dispatch<MOE_DT_F32, MOE_DT_F32>(k, vec, s);
  else if (BT == MOE_DT_BF16) e = dispatch<MOE_DT_F32, MOE_DT_BF16>(k, vec, s);
  else e = dispatch<MOE_DT_F32, MOE_DT_F16>(k, vec, s);
  return launch_status(e);
}
