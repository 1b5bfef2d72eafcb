// The norms around a block, fused with its gate and its residual (forward and backward).
//
//   a = y SiLU(z);  p = a r w_post, r = 1 / sqrt(mean_group(a²) + eps);  h = α res + β p;
//   n = h r_h w_pre, r_h = 1 / sqrt(mean(h²) + eps)          (gate_last: p = y r w_post SiLU(z))
// ("Mamba y las SSMs", "Mamba" (Figura 3: the gated SSM) and "Estado interno puramente lineal" (output
// projection and residual connection); the pages leave the norms out.)
//
// Backward, with ĥ = h r_h and â = a r:
//   dh = g_h + r_h (g_n w_pre - ĥ mean(g_n w_pre ĥ));  dres = α dh;  dp = β dh
//   da = r (dp w_post - â mean_group(dp w_post â));  dy = da SiLU(z);  dz = da y SiLU'(z)
//   dw_pre = Σ_rows g_n ĥ;  dw_post = Σ_rows dp â
// The forward is computed again from y, z and res, so nothing but its inputs is kept for training and
// the gradients do not see h's rounding.
//
// Bound by memory: every tensor is read or written once, 16 bytes per thread and access. A row is held
// in registers, 8-channel vectors dealt to its TPR threads in turn, so that each pass over the row
// after the first costs no memory. All sums are fp32 and taken in a fixed order.
#include <algorithm>

#include "common.cuh"

namespace swimba {
swimba_status api_cuda_status(cudaError_t e);

namespace {

constexpr int kMaxWidth = 16384;
constexpr int kSMs = 148;

struct NormParams {
  const void *y, *z, *res, *g_h, *g_n;
  const float *w_post, *w_pre;
  void *h, *n;              // forward
  void *dy, *dz, *dres;     // backward
  float* part;              // backward: [CTAs][2][width] partial sums of dw_post and dw_pre
  int64_t rows;
  int width, groups, gate_last;
  float eps, alpha, beta;
};

// 8 consecutive values of a row.
template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  const T* p = reinterpret_cast<const T*>(base) + at;
  if constexpr (sizeof(T) == 2) {
    Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(p), v);
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&v)[8]) {
  T* p = reinterpret_cast<T*>(base) + at;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

template <int TPR>
__device__ __forceinline__ void row_sync() {
  if constexpr (TPR == 32) __syncwarp();
  else __syncthreads();
}

// Sums of K values over the TPR threads of a row, the same in every thread. `red`: 32 K floats of shared
// memory that no other sum of this row uses between two row_syncs.
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = lane < TPR / 32 ? red[k * 32 + lane] : 0.f;
#pragma unroll
      for (int o = TPR / 64; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[k] = __shfl_sync(0xffffffffu, s, 0);
    }
  }
}

// Sums over the groups of a row: v[i] is this thread's sum over its vector i, and becomes the sum over
// the group that the vector lies in. Groups of 8, 16 .. 256 channels in powers of two are whole aligned
// sets of lanes and meet in shuffles; others go through shared memory (`gred`: a float per vector and
// one per group), one warp per group.
template <int TPR, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], int nvec, int groups, int tid, float* red, float* gred) {
  if (groups == 1) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) s[0] += v[i];
    row_sum<TPR, 1>(s, red);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = s[0];
    return;
  }
  const int gv = nvec / groups;
  if (gv <= 32 && (gv & (gv - 1)) == 0) {
    for (int o = gv >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    return;
  }
  float* gsum = gred + nvec;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + i * TPR < nvec) gred[tid + i * TPR] = v[i];
  row_sync<TPR>();
  const int lane = tid & 31;
  for (int g = tid >> 5; g < groups; g += TPR / 32) {
    float s = 0.f;
    for (int j = lane; j < gv; j += 32) s += gred[g * gv + j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) gsum[g] = s;
  }
  row_sync<TPR>();
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + i * TPR < nvec) v[i] = gsum[(tid + i * TPR) / gv];
}

// Dynamic shared memory of a row: the cross-warp sums and, for groups that need it, group_sum's.
__device__ __forceinline__ float* row_smem(float* base, int slot, int nvec, int groups) {
  return base + (size_t)slot * (3 * 64 + nvec + groups);
}

// ---- forward ---------------------------------------------------------------------------------------------
template <typename IO, typename RES, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_fwd_kernel(const NormParams p) {
  extern __shared__ float smem[];
  constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
  const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + slot;
  if (row >= p.rows) return;  // a whole warp, or the whole CTA
  const int nvec = p.width / 8;
  float* red = row_smem(smem, slot, nvec, p.groups);
  float* gred = red + 3 * 64;
  float a[NV][8], gate[NV][8];
  const int64_t base = row * p.width;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * TPR;
#pragma unroll
    for (int e = 0; e < 8; ++e) a[i][e] = 0.f, gate[i][e] = 0.f;
    if (v >= nvec) continue;
    if (p.y) load8<IO>(p.y, base + 8 * v, a[i]);
    if (p.z) load8<IO>(p.z, base + 8 * v, gate[i]);
  }
  if (p.z) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        gate[i][e] *= sigmoid(gate[i][e]);
        if (!p.gate_last) a[i][e] *= gate[i][e];
      }
  }
  if (p.w_post) {
    float s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i] = fmaf(a[i][e], a[i][e], s[i]);
    }
    group_sum<TPR, NV>(s, nvec, p.groups, tid, red, gred);
    const float inv = (float)p.groups / (float)p.width;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * TPR;
      if (v >= nvec) continue;
      const float r = rsqrtf(fmaf(s[i], inv, p.eps));
      float w[8];
      load8<float>(p.w_post, 8 * v, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i][e] *= r * w[e];
    }
  }
  if (p.z && p.gate_last) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i][e] *= gate[i][e];
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * TPR;
    if (v >= nvec) continue;
    float r[8] = {};
    if (p.res) load8<RES>(p.res, base + 8 * v, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[i][e] = p.res ? fmaf(p.alpha, r[e], p.beta * a[i][e]) : p.beta * a[i][e];
      ss[0] = fmaf(a[i][e], a[i][e], ss[0]);
    }
    if (p.h) store8<RES>(p.h, base + 8 * v, a[i]);
  }
  if (p.n == nullptr) return;
  row_sum<TPR, 1>(ss, red + 64);
  const float r = rsqrtf(ss[0] / (float)p.width + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * TPR;
    if (v >= nvec) continue;
    float w[8];
    load8<float>(p.w_pre, 8 * v, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[i][e] *= r * w[e];
    store8<IO>(p.n, base + 8 * v, a[i]);
  }
}

// ---- backward --------------------------------------------------------------------------------------------
// A CTA walks rows blockIdx.x, blockIdx.x + gridDim.x, ..., keeps its threads' columns of the two
// weight gradients in registers and writes them once, to be summed over the CTAs by norm_dw_kernel.
template <typename IO, typename RES, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_bwd_kernel(const NormParams p) {
  extern __shared__ float smem[];
  constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
  const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int nvec = p.width / 8;
  float* red = row_smem(smem, slot, nvec, p.groups);
  float* gred = red + 3 * 64;
  float dwp[NV][8], dwn[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dwp[i][e] = 0.f, dwn[i][e] = 0.f;
  const float inv = 1.f / (float)p.width, ginv = (float)p.groups / (float)p.width;
  for (int64_t row = (int64_t)blockIdx.x * RPB + slot; row < p.rows; row += (int64_t)gridDim.x * RPB) {
    const int64_t base = row * p.width;
    float y[NV][8], z[NV][8], hat[NV][8], dh[NV][8], h[NV][8], gn[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * TPR;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = z[i][e] = dh[i][e] = h[i][e] = gn[i][e] = 0.f;
      if (v >= nvec) continue;
      if (p.y) load8<IO>(p.y, base + 8 * v, y[i]);
      if (p.z) load8<IO>(p.z, base + 8 * v, z[i]);
      if (p.res) load8<RES>(p.res, base + 8 * v, h[i]);
      if (p.g_h) load8<RES>(p.g_h, base + 8 * v, dh[i]);
      if (p.g_n) load8<IO>(p.g_n, base + 8 * v, gn[i]);
    }
    // the forward: a, its norm, h
    float r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hat[i][e] = (p.z && !p.gate_last) ? y[i][e] * (z[i][e] * sigmoid(z[i][e])) : y[i][e];
        r[i] = fmaf(hat[i][e], hat[i][e], r[i]);
      }
    }
    if (p.w_post) {
      group_sum<TPR, NV>(r, nvec, p.groups, tid, red, gred);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        r[i] = rsqrtf(fmaf(r[i], ginv, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) hat[i][e] *= r[i];
      }
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * TPR;
      if (v >= nvec) continue;
      float wp[8], wn[8];
      if (p.w_post) load8<float>(p.w_post, 8 * v, wp);
      if (p.g_n) load8<float>(p.w_pre, 8 * v, wn);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float q = p.w_post ? hat[i][e] * wp[e] : hat[i][e];
        if (p.z && p.gate_last) q *= z[i][e] * sigmoid(z[i][e]);
        h[i][e] = fmaf(p.alpha, h[i][e], p.beta * q);
        if (p.g_n) {
          s[0] = fmaf(h[i][e], h[i][e], s[0]);
          s[1] = fmaf(gn[i][e] * wn[e], h[i][e], s[1]);
        }
      }
    }
    if (p.g_n) {
      row_sum<TPR, 2>(s, red + 64);
      const float rh = rsqrtf(fmaf(s[0], inv, p.eps)), m = s[1] * rh * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * TPR;
        if (v >= nvec) continue;
        float wn[8];
        load8<float>(p.w_pre, 8 * v, wn);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float hh = h[i][e] * rh;
          dwn[i][e] = fmaf(gn[i][e], hh, dwn[i][e]);
          dh[i][e] = fmaf(rh, fmaf(-hh, m, gn[i][e] * wn[e]), dh[i][e]);
        }
      }
    }
    // back through the residual, the gate behind the norm, the norm
    float q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * TPR;
      q[i] = 0.f;
      if (v >= nvec) continue;
      if (p.dres) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = p.alpha * dh[i][e];
        store8<RES>(p.dres, base + 8 * v, d);
      }
      float wp[8], dz[8];
      if (p.w_post) load8<float>(p.w_post, 8 * v, wp);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float d = p.beta * dh[i][e];
        if (p.z && p.gate_last) {
          const float sg = sigmoid(z[i][e]);
          dz[e] = d * (p.w_post ? hat[i][e] * wp[e] : hat[i][e]) * (sg * fmaf(z[i][e], 1.f - sg, 1.f));
          d *= z[i][e] * sg;
        }
        if (p.w_post) {
          dwp[i][e] = fmaf(d, hat[i][e], dwp[i][e]);
          d *= wp[e];
          q[i] = fmaf(d, hat[i][e], q[i]);
        }
        dh[i][e] = d;
      }
      if (p.z && p.gate_last) store8<IO>(p.dz, base + 8 * v, dz);
    }
    if (p.w_post) group_sum<TPR, NV>(q, nvec, p.groups, tid, red + 128, gred);
    if (p.y) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * TPR;
        if (v >= nvec) continue;
        float dz[8];
        const float m = q[i] * ginv;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float d = p.w_post ? r[i] * fmaf(-hat[i][e], m, dh[i][e]) : dh[i][e];
          if (p.z && !p.gate_last) {
            const float sg = sigmoid(z[i][e]);
            dz[e] = d * y[i][e] * (sg * fmaf(z[i][e], 1.f - sg, 1.f));
            d *= z[i][e] * sg;
          }
          dh[i][e] = d;
        }
        store8<IO>(p.dy, base + 8 * v, dh[i]);
        if (p.z && !p.gate_last) store8<IO>(p.dz, base + 8 * v, dz);
      }
    }
    row_sync<TPR>();  // the shared sums are free for the next row
  }
  if (p.part == nullptr) return;
  // this CTA's sums; a CTA's row slots add up one after the other
  float* part = p.part + (size_t)blockIdx.x * 2 * p.width;
  for (int k = 0; k < RPB; ++k) {
    if (k == slot) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * TPR;
        if (v >= nvec) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float* d = part + (size_t)w * p.width + 8 * v;
          const float(&a)[8] = w ? dwn[i] : dwp[i];
          float o[8] = {};
          if (k > 0) load8<float>(d, 0, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += a[e];
          store8<float>(d, 0, o);
        }
      }
    }
    if (RPB > 1) __syncthreads();
  }
}

// dw[c] = Σ over CTAs of part[cta][which][c]: 8 threads per column, each every eighth CTA.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* part, int ctas, int width, float* dw_post, float* dw_pre) {
  __shared__ float red[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5, which = blockIdx.y;
  float* out = which ? dw_pre : dw_post;
  if (out == nullptr) return;
  float s = 0.f;
  if (c < width)
    for (int i = k; i < ctas; i += 8) s += part[((size_t)i * 2 + which) * width + c];
  red[k][threadIdx.x & 31] = s;
  __syncthreads();
  if (k == 0 && c < width) {
    for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
    out[c] = s;
  }
}

// ---- host ------------------------------------------------------------------------------------------------

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

swimba_status check_norm(const swimba_norm_dims* d) {
  if (d == nullptr || d->rows <= 0 || d->width <= 0 || d->groups <= 0 || !(d->eps > 0.f)) return SWIMBA_ERR_INVALID_ARG;
  if ((d->io_dtype != SWIMBA_F32 && d->io_dtype != SWIMBA_BF16) ||
      (d->res_dtype != SWIMBA_F32 && d->res_dtype != SWIMBA_BF16) || (d->gate_last != 0 && d->gate_last != 1))
    return SWIMBA_ERR_INVALID_ARG;
  if (d->width % 8 || d->width > kMaxWidth || d->width % d->groups || (d->width / d->groups) % 8)
    return SWIMBA_ERR_UNSUPPORTED;
  if (d->rows > (int64_t(1) << 31)) return SWIMBA_ERR_UNSUPPORTED;
  return SWIMBA_OK;
}

// Threads per row: enough that a thread holds at most two vectors of 8 channels (four below 1024
// channels, where a warp then needs no barrier).
int threads_per_row(int width) {
  const int nvec = width / 8;
  return nvec <= 128 ? 32 : nvec <= 256 ? 128 : nvec <= 512 ? 256 : nvec <= 1024 ? 512 : 1024;
}

// CTAs of the backward: up to two resident per SM, so that one's loads cover another's sums.
int bwd_ctas(const swimba_norm_dims* d) {
  const int tpr = threads_per_row(d->width), rpb = tpr < 128 ? 128 / tpr : 1;
  return (int)std::min<int64_t>((d->rows + rpb - 1) / rpb, tpr >= 512 ? kSMs : 2 * kSMs);
}

size_t row_smem_bytes(const swimba_norm_dims* d, int rpb) {
  return (size_t)rpb * (3 * 64 + d->width / 8 + d->groups) * sizeof(float);
}

template <typename IO, typename RES, int TPR, int NV>
cudaError_t launch_norm(const swimba_norm_dims* d, const NormParams& p, bool bwd, cudaStream_t s) {
  constexpr int RPB = TPR < 128 ? 128 / TPR : 1, T = TPR < 128 ? 128 : TPR;
  const size_t smem = row_smem_bytes(d, RPB);
  if (bwd) {
    norm_bwd_kernel<IO, RES, TPR, NV><<<(unsigned)bwd_ctas(d), T, smem, s>>>(p);
  } else {
    norm_fwd_kernel<IO, RES, TPR, NV><<<(unsigned)((d->rows + RPB - 1) / RPB), T, smem, s>>>(p);
  }
  note_launch();
  return cudaGetLastError();
}

template <typename IO, typename RES>
cudaError_t run_norm(const swimba_norm_dims* d, const NormParams& p, bool bwd, cudaStream_t s) {
  const int nvec = d->width / 8;
  switch (threads_per_row(d->width)) {
    case 32:
      return nvec <= 32   ? launch_norm<IO, RES, 32, 1>(d, p, bwd, s)
             : nvec <= 64 ? launch_norm<IO, RES, 32, 2>(d, p, bwd, s)
                          : launch_norm<IO, RES, 32, 4>(d, p, bwd, s);
    case 128: return launch_norm<IO, RES, 128, 2>(d, p, bwd, s);
    case 256: return launch_norm<IO, RES, 256, 2>(d, p, bwd, s);
    case 512: return launch_norm<IO, RES, 512, 2>(d, p, bwd, s);
    default: return launch_norm<IO, RES, 1024, 2>(d, p, bwd, s);
  }
}

cudaError_t run_norm_types(const swimba_norm_dims* d, const NormParams& p, bool bwd, cudaStream_t s) {
  const bool io = d->io_dtype == SWIMBA_BF16, res = d->res_dtype == SWIMBA_BF16;
  if (io) return res ? run_norm<__nv_bfloat16, __nv_bfloat16>(d, p, bwd, s) : run_norm<__nv_bfloat16, float>(d, p, bwd, s);
  return res ? run_norm<float, __nv_bfloat16>(d, p, bwd, s) : run_norm<float, float>(d, p, bwd, s);
}

NormParams norm_params(const swimba_norm_dims* d, const void* y, const void* z, const float* w_post, const void* res,
                       const float* w_pre) {
  NormParams p{};
  p.y = y;
  p.z = z;
  p.res = res;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.rows = d->rows;
  p.width = d->width;
  p.groups = d->groups;
  p.gate_last = d->gate_last;
  p.eps = d->eps;
  p.alpha = d->res_scale;
  p.beta = d->out_scale;
  return p;
}

bool parts_ok(const void* y, const void* z, const float* w_post, const void* res) {
  return y != nullptr || (z == nullptr && w_post == nullptr && res != nullptr);
}

}  // namespace
}  // namespace swimba

using namespace swimba;

extern "C" {

swimba_status swimba_block_norm_fwd(const swimba_norm_dims* dims, const void* y, const void* z, const float* w_post,
                                    const void* res, const float* w_pre, void* h, void* n, void* stream) {
  const swimba_status st = check_norm(dims);
  if (st != SWIMBA_OK) return st;
  if (!parts_ok(y, z, w_post, res) || (!h && !n) || (n != nullptr) != (w_pre != nullptr) || (n && n == h))
    return SWIMBA_ERR_INVALID_ARG;
  if ((h && (h == y || h == z)) || (n && n == res)) return SWIMBA_ERR_INVALID_ARG;
  if (!aligned16(y) || !aligned16(z) || !aligned16(w_post) || !aligned16(res) || !aligned16(w_pre) || !aligned16(h) ||
      !aligned16(n))
    return SWIMBA_ERR_ALIGN;
  NormParams p = norm_params(dims, y, z, w_post, res, w_pre);
  p.h = h;
  p.n = n;
  return api_cuda_status(run_norm_types(dims, p, false, static_cast<cudaStream_t>(stream)));
}

size_t swimba_block_norm_workspace_size(const swimba_norm_dims* dims) {
  if (check_norm(dims) != SWIMBA_OK) return 0;
  return kStatusBytes + (size_t)bwd_ctas(dims) * 2 * dims->width * sizeof(float);
}

swimba_status swimba_block_norm_bwd(const swimba_norm_dims* dims, const void* y, const void* z, const float* w_post,
                                    const void* res, const float* w_pre, const void* g_h, const void* g_n, void* dy,
                                    void* dz, void* dres, float* dw_post, float* dw_pre, void* ws, size_t ws_bytes,
                                    void* stream) {
  const swimba_status st = check_norm(dims);
  if (st != SWIMBA_OK) return st;
  auto differ = [](const void* a, const void* b) { return (a != nullptr) != (b != nullptr); };
  if (!parts_ok(y, z, w_post, res) || differ(y, dy) || differ(z, dz) || differ(res, dres) || differ(w_post, dw_post) ||
      differ(w_pre, dw_pre) || differ(w_pre, g_n) || (!g_h && !g_n))
    return SWIMBA_ERR_INVALID_ARG;
  if (ws == nullptr || ws_bytes < swimba_block_norm_workspace_size(dims)) return SWIMBA_ERR_WORKSPACE;
  if (!aligned16(y) || !aligned16(z) || !aligned16(w_post) || !aligned16(res) || !aligned16(w_pre) || !aligned16(g_h) ||
      !aligned16(g_n) || !aligned16(dy) || !aligned16(dz) || !aligned16(dres) || !aligned16(dw_post) ||
      !aligned16(dw_pre) || !aligned16(ws))
    return SWIMBA_ERR_ALIGN;
  NormParams p = norm_params(dims, y, z, w_post, res, w_pre);
  p.g_h = g_h;
  p.g_n = g_n;
  p.dy = dy;
  p.dz = dz;
  p.dres = dres;
  const bool weights = w_post || w_pre;
  p.part = weights ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = run_norm_types(dims, p, true, s);
  if (e != cudaSuccess || !weights) return api_cuda_status(e);
  norm_dw_kernel<<<dim3((unsigned)((dims->width + 31) / 32), 2), 256, 0, s>>>(p.part, bwd_ctas(dims), dims->width, dw_post,
                                                                             dw_pre);
  note_launch();
  return api_cuda_status(cudaGetLastError());
}

}  // extern "C"
