// Linear attention with a decay for each head: C ABI entry points, the fp32 recurrence, the decode
// step and the small kernels around them (segment chain, shared-head sums, zero rows).
//
// Sources: "Swimba: Switch Mamba Model Scales State Space Models", Dutch summary §2 "Architectuur
// Implementatie" (the chunked processing of the state space dual form carries over) and "Mamba y las
// SSMs", "Estado interno puramente lineal" (a linear state can be cut into pieces and recombined);
// the recurrence itself is stated in include/swimba.h.
#include <algorithm>
#include <cstdio>
#include <type_traits>

#include "linattn.cuh"

namespace swimba {
swimba_status api_cuda_status(cudaError_t e);
cudaError_t run_la_tc(const LaParams& p, bool states, cudaStream_t s);

namespace {

constexpr int kSimtTokens = 16;   // tokens staged per step
constexpr int kSimtCols = 64;     // columns of M per CTA
constexpr int kSMs = 148;

template <typename IO>
__device__ __forceinline__ const IO* la_row(const LaStream& s, int b, int64_t t, int h, int d) {
  return reinterpret_cast<const IO*>(s.p) + b * s.sb + t * s.st + (int64_t)(h / s.div) * d;
}

// ---- the recurrence, token by token ------------------------------------------------------------------
// One CTA of 128 threads per (role, sequence, head, segment, 64 columns of M). A thread keeps NI x 4
// rows (16 i + 4 p + 0..3, p its quarter) of two columns in registers, so a token costs it 3 FMA-pipe
// operations per state element and one 16-byte shared read of x and of y per 8 of them; the four
// quarters' partial readouts meet in two shuffles. Bound by the FMA pipe (3 d_x d_w operations per
// token and head, 2 where decays are put off). MODE 0 writes the outputs, MODE 1 only the segment's end state from zero.
// (A count of 4 CTAs for NI = 8 gives it a better order of instructions too: 4 x 1024 tokens of 16 heads backward 920
// -> 886 us; counts for the others, with their spills or fewer CTAs, cost them up to 40 %.)
template <typename IO, int NI, int MODE>
__global__ void __launch_bounds__(128, NI == 8 ? 4 : 0) la_simt_kernel(const __grid_constant__ LaParams p) {
  __shared__ __align__(16) float sx[kSimtTokens][NI * 16];
  __shared__ __align__(16) float sy[kSimtTokens][NI * 16];
  __shared__ __align__(16) float sw[kSimtTokens][kSimtCols];
  __shared__ __align__(16) float so[MODE == 0 ? kSimtTokens : 1][kSimtCols];
  __shared__ float later[kSimtTokens + 1], sooner[kSimtTokens + 1];  // γ^e and γ^-e
  __shared__ float one, slip;                                        // γ and its relative error
  __shared__ LaDecay all;                                            // γ^kSimtTokens
  const int tid = threadIdx.x, lane = tid & 31, part = lane & 3;
  const int col = (tid >> 5) * 16 + (lane >> 2) * 2;
  int64_t item = blockIdx.x;
  const int seg = (int)(item % p.nseg);
  item /= p.nseg;
  const int64_t bh = item % ((int64_t)p.B * p.H);
  const LaRole& r = p.role[item / ((int64_t)p.B * p.H)];
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int c_base = blockIdx.y * kSimtCols;
  if (c_base >= r.dw) return;
  const int ncol = min(kSimtCols, r.dw - c_base);
  // γ's rounding would grow with every token that a state outlives: `slip`, its relative error, is taken out
  // of the state after every kSimtTokens tokens (without it 4e-6 in place of 3e-7 at 333 tokens).
  // Where γ is so near 1 that kSimtTokens tokens take less than 40 % of a state (`lazy`), they leave M as it is, their
  // values enter it times γ^-e and their readouts leave it times γ^e, and then it decays once, by γ^kSimtTokens's hi
  // or hi ± 2^-24 as in the tensor-core kernel: a product with γ at every token would be rounded in one direction
  // (16384 tokens at log decays of -2^-17 to -2^-24: 6e-6 in place of 5e-7).
  const float g = p.g[h];
  const bool lazy = fabsf(g) * kSimtTokens < 0.5f;
  if (tid < 64 && lane <= kSimtTokens) {
    const bool back = tid >= 32;
    const double e = exp((double)g * (back ? -lane : lane));
    const LaDecay d = {(float)e, (float)(e - (double)(float)e)};
    (back ? sooner : later)[lane] = d.hi;
    if (!back && lane == 1) one = d.hi, slip = d.hi > 0.f ? d.lo / d.hi : 0.f;
    if (!back && lane == kSimtTokens) all = d;
  }
  __syncthreads();
  const float gamma = one, slip1 = slip;
  const int64_t len = la_len(p, b);
  int c0, c1;
  la_segment(p, len, seg, r.rev, c0, c1);
  const int64_t lo = (int64_t)c0 * p.chunk, hi = min((int64_t)c1 * p.chunk, len);

  float M[NI * 4][2];
  const float* start = p.nseg > 1 ? r.seg + (bh * p.nseg + seg) * r.dx * r.dw : r.M0 ? r.M0 + bh * r.dx * r.dw : nullptr;
  const int sj = p.nseg > 1 ? r.dw : r.sj, sc = p.nseg > 1 ? 1 : r.sc;
#pragma unroll
  for (int i = 0; i < NI * 4; ++i) {
    const int j = 16 * (i >> 2) + 4 * part + (i & 3);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      M[i][e] = (MODE == 0 && start != nullptr && j < r.dx && col + e < ncol)
                    ? start[(int64_t)j * sj + (int64_t)(c_base + col + e) * sc]
                    : 0.f;
  }
  for (int i = tid; i < kSimtTokens * NI * 16; i += 128) {  // the padding stays zero
    sx[0][i] = 0.f;
    sy[0][i] = 0.f;
  }
  for (int i = tid; i < kSimtTokens * kSimtCols; i += 128) sw[0][i] = 0.f;

  constexpr int V = Vec16<IO>::n;
  for (int64_t at = 0; at < hi - lo; at += kSimtTokens) {
    const int n = (int)min((int64_t)kSimtTokens, hi - lo - at);
    const int before = r.rev && at == 0 ? 0 : 1;  // decays before the first token: a reverse segment's M has had it
    auto token = [&](int i) { return r.rev ? hi - 1 - at - i : lo + at + i; };
    __syncthreads();
    auto stage = [&](const LaStream& s, float* dst, int pitch, int first, int count, int d, float scale, bool value) {
      const int per = count / V;
      for (int i = tid; i < n * per; i += 128) {
        const int t = i / per, v = (i - t * per) * V;
        const float f = value && lazy ? scale * sooner[t + before] : scale;
        float f8[V];
        Vec16<IO>::unpack(*reinterpret_cast<const uint4*>(la_row<IO>(s, b, token(t), h, d) + first + v), f8);
#pragma unroll
        for (int e = 0; e < V; ++e) dst[t * pitch + v + e] = f8[e] * f;
      }
    };
    if (MODE == 0) stage(r.x, sx[0], NI * 16, 0, r.dx, r.dx, 1.f, false);
    stage(r.y, sy[0], NI * 16, 0, r.dx, r.dx, 1.f, false);
    stage(r.w, sw[0], kSimtCols, c_base, ncol, r.dw, r.s_u, true);
    __syncthreads();
    float decay = before ? gamma : 1.f;
    if (!lazy) {
      const float slip_n = slip1 * (float)n;
#pragma unroll
      for (int i = 0; i < NI * 4; ++i) {
        M[i][0] = fmaf(M[i][0], slip_n, M[i][0]);
        M[i][1] = fmaf(M[i][1], slip_n, M[i][1]);
      }
    }
    auto tokens = [&](auto put_off) {
      for (int t = 0; t < n; ++t) {
        const float2 w = *reinterpret_cast<const float2*>(&sw[t][col]);
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(&sy[t][16 * i + 4 * part]);
          const float yv[4] = {y.x, y.y, y.z, y.w};
          float xv[4] = {};
          if (MODE == 0) {
            const float4 x = *reinterpret_cast<const float4*>(&sx[t][16 * i + 4 * part]);
            xv[0] = x.x, xv[1] = x.y, xv[2] = x.z, xv[3] = x.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* m = M[4 * i + e];
            m[0] = fmaf(yv[e], w.x, put_off ? m[0] : m[0] * decay);
            m[1] = fmaf(yv[e], w.y, put_off ? m[1] : m[1] * decay);
            if (MODE == 0) {
              a0 = fmaf(xv[e], m[0], a0);
              a1 = fmaf(xv[e], m[1], a1);
            }
          }
        }
        decay = gamma;
        if (MODE == 0) {
          a0 += __shfl_xor_sync(0xffffffffu, a0, 1);
          a1 += __shfl_xor_sync(0xffffffffu, a1, 1);
          a0 += __shfl_xor_sync(0xffffffffu, a0, 2);
          a1 += __shfl_xor_sync(0xffffffffu, a1, 2);
          const float f = put_off ? r.s_inter * later[t + before] : r.s_inter;
          if (part == 0) *reinterpret_cast<float2*>(&so[t][col]) = make_float2(a0 * f, a1 * f);
        }
      }
    };
    if (!lazy) {
      tokens(std::false_type{});
    } else {
      tokens(std::true_type{});
      const int e = n - 1 + before;
      const float f = e == kSimtTokens ? la_factor(all, (int)(at / kSimtTokens)) : later[e];
#pragma unroll
      for (int i = 0; i < NI * 4; ++i) {
        M[i][0] *= f;
        M[i][1] *= f;
      }
    }
    if (MODE == 0) {
      __syncthreads();
      for (int i = tid; i < n * ncol; i += 128) {
        const int t = i / ncol, c = i - t * ncol;
        const int64_t at_out = b * r.out_sb + token(t) * r.out_st + (int64_t)h * r.dw + c_base + c;
        if (r.out_f32) reinterpret_cast<float*>(r.out)[at_out] = so[t][c];
        else from_f32(reinterpret_cast<IO*>(r.out)[at_out], so[t][c]);
      }
    }
  }
  if (MODE == 0 && (p.nseg > 1 || r.M_end == nullptr)) return;
  // a reverse segment leaves M decayed to the token before it
  const float last = r.rev && hi > lo ? one : 1.f;
  float* end = MODE == 1 ? r.seg + (bh * p.nseg + seg) * r.dx * r.dw : r.M_end + bh * r.dx * r.dw;
  const int ej = MODE == 1 ? r.dw : r.sj, ec = MODE == 1 ? 1 : r.sc;
#pragma unroll
  for (int i = 0; i < NI * 4; ++i) {
    const int j = 16 * (i >> 2) + 4 * part + (i & 3);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (j < r.dx && col + e < ncol) end[(int64_t)j * ej + (int64_t)(c_base + col + e) * ec] = M[i][e] * last;
  }
}

// ---- segment chain -------------------------------------------------------------------------------------
// seg[s] holds segment s's end state from zero; it becomes the state before segment s, and the state
// after the last one goes to M_end. One thread per 4 elements of a row, their segments' states loaded
// kBatch at a time (the stores in between would keep the compiler from moving the loads up).
__global__ void __launch_bounds__(128) la_chain_kernel(const __grid_constant__ LaParams p) {
  constexpr int kBatch = 8;
  const uint32_t bhs = (uint32_t)p.B * p.H, item = blockIdx.x;
  const LaRole& r = p.role[item / bhs];
  const uint32_t bh = item % bhs;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H), dw = r.dw, size = r.dx * dw, rev = r.rev, nseg = p.nseg;
  const int e = (blockIdx.y * 128 + threadIdx.x) * 4;
  if (e >= size) return;
  const int j = e / dw, c = e - j * dw, sj = r.sj, sc = r.sc;
  const LaDecay g_all = la_decay(p.g[h], p.cps * p.chunk);
  const int64_t len = la_len(p, b);
  float4* seg = reinterpret_cast<float4*>(r.seg + (int64_t)bh * nseg * size + e);
  const int64_t own = (int64_t)bh * size + (int64_t)j * sj + (int64_t)c * sc;
  const float* M0 = r.M0;
  float* M_end = r.M_end;
  float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M0) m = make_float4(M0[own], M0[own + sc], M0[own + 2 * sc], M0[own + 3 * sc]);
  for (int s0 = 0; s0 < nseg; s0 += kBatch) {
    float4 end[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (s0 + i < nseg) end[i] = seg[(int64_t)(s0 + i) * (size / 4)];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i < nseg) {
        int c0, c1;
        la_segment(p, len, s0 + i, rev, c0, c1);
        const int n = (int)(min((int64_t)c1 * p.chunk, len) - min((int64_t)c0 * p.chunk, len));
        seg[(int64_t)(s0 + i) * (size / 4)] = m;
        if (n > 0) {
          const LaDecay g = n == p.cps * p.chunk ? g_all : la_decay(p.g[h], n);
          m.x = fmaf(g.hi, m.x, fmaf(g.lo, m.x, end[i].x));
          m.y = fmaf(g.hi, m.y, fmaf(g.lo, m.y, end[i].y));
          m.z = fmaf(g.hi, m.z, fmaf(g.lo, m.z, end[i].z));
          m.w = fmaf(g.hi, m.w, fmaf(g.lo, m.w, end[i].w));
        }
      }
    }
  }
  if (M_end) {
    M_end[own] = m.x;
    M_end[own + sc] = m.y;
    M_end[own + 2 * sc] = m.z;
    M_end[own + 3 * sc] = m.w;
  }
}

// ---- rows without a token, shared heads ----------------------------------------------------------------
// out[b, t, kv, :] = Σ_i part[b, t, kv group + i, :] for tokens inside the sequence (fixed order), zeros
// in the rows behind it; with part == null only the zeros are written. One thread per 8 elements.
struct LaRowsOf {
  void* out;
  int64_t st;         // elements from one token to the next
  const float* part;  // [rows, heads, group, d], or null: only zeros behind the sequences' ends
  int heads, d;
};
struct LaRows {
  LaRowsOf of[3];
  const int32_t* lens;  // or null
  int64_t B, L;
  int group;
};
template <typename IO>
__global__ void __launch_bounds__(256) la_rows_kernel(const __grid_constant__ LaRows p) {
  const LaRowsOf& r = p.of[blockIdx.y];
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int width = r.heads * r.d, per = width / 8;
  const int64_t row = i / per, b = row / p.L, t = row - b * p.L;
  if (b >= p.B) return;
  const int at = (int)(i - row * per) * 8;
  const bool live = p.lens == nullptr || t < (int64_t)p.lens[b];
  if (live && r.part == nullptr) return;
  float v[8] = {};
  if (live) {
    const int kv = at / r.d, j = at - kv * r.d;
    const float* src = r.part + (row * width + (int64_t)kv * r.d) * p.group + j;
    for (int g = 0; g < p.group; ++g) {
      const float4 a = *reinterpret_cast<const float4*>(src + g * r.d), c = *reinterpret_cast<const float4*>(src + g * r.d + 4);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      v[4] += c.x, v[5] += c.y, v[6] += c.z, v[7] += c.w;
    }
  }
  IO* dst = reinterpret_cast<IO*>(r.out) + row * r.st + at;
  if constexpr (sizeof(IO) == 2) {
    __align__(16) IO x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) from_f32(x[e], v[e]);
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(x);
  } else {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// ---- decode step ----------------------------------------------------------------------------------------
// One CTA per (sequence, head) and `cols` columns: the state is read and written once (8 d_k d_v bytes),
// which bounds it: 512 MiB of state, bf16 tokens, in 163 us, the measured copy rate. Threads go over the state
// row by row, 16 bytes each; the partial readouts of the threads that share columns meet in shared memory.
// Few heads are cut into 32 columns (128 bytes of a row), so that every SM has a share: 96 heads of 128 x 128
// take 4.1 us, 6.2 whole. Many heads stay whole, rows of 512 bytes; a call of a few heads is bound by its launch.
template <typename IO>
__global__ void __launch_bounds__(256) la_step_kernel(LaStream q, LaStream k, LaStream v, const float* g,
                                                      const float* S_in, IO* o, float* S_out, int H, int dk, int dv,
                                                      int cols, float scale) {
  __shared__ float sq[128], sk[128];
  __shared__ LaDecay decay;
  __shared__ __align__(16) float red[1024];
  const int64_t bh = blockIdx.x;
  const int b = (int)(bh / H), h = (int)(bh % H), tid = threadIdx.x, first = blockIdx.y * cols;
  const int mine = min(cols, dv - first), c4 = mine / 4, R = 256 / c4, r0 = tid / c4, c = tid - r0 * c4, pitch = dv / 4;
  const float4* in = reinterpret_cast<const float4*>(S_in + bh * dk * dv + first) + c;
  float4* out = reinterpret_cast<float4*>(S_out + bh * dk * dv + first) + c;
  if (tid < dk) {
    sq[tid] = to_f32(la_row<IO>(q, b, 0, h, dk)[tid]) * scale;
    sk[tid] = to_f32(la_row<IO>(k, b, 0, h, dk)[tid]);
  }
  if (tid == 255) decay = la_decay(g[h], 1);  // (in every thread, 64 x 32 heads of 64 x 64 took 22.2 us in place of 21.4)
  __syncthreads();
  const LaDecay gamma = decay;
  if (r0 < R) {
    const IO* vp = la_row<IO>(v, b, 0, h, dv) + first + 4 * c;
    const float4 vv = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;  // rows in flight
    for (int j0 = r0; j0 < dk; j0 += kBatch * R) {
      float4 s[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (j0 + i * R < dk) s[i] = in[(int64_t)(j0 + i * R) * pitch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = j0 + i * R;
        if (j >= dk) break;
        const float kj = sk[j], qj = sq[j];
        s[i].x = fmaf(gamma.hi, s[i].x, fmaf(gamma.lo, s[i].x, kj * vv.x));
        s[i].y = fmaf(gamma.hi, s[i].y, fmaf(gamma.lo, s[i].y, kj * vv.y));
        s[i].z = fmaf(gamma.hi, s[i].z, fmaf(gamma.lo, s[i].z, kj * vv.z));
        s[i].w = fmaf(gamma.hi, s[i].w, fmaf(gamma.lo, s[i].w, kj * vv.w));
        acc.x = fmaf(qj, s[i].x, acc.x);
        acc.y = fmaf(qj, s[i].y, acc.y);
        acc.z = fmaf(qj, s[i].z, acc.z);
        acc.w = fmaf(qj, s[i].w, acc.w);
        out[(int64_t)j * pitch] = s[i];
      }
    }
    reinterpret_cast<float4*>(red)[r0 * c4 + c] = acc;
  }
  __syncthreads();
  if (tid < mine) {
    float a = 0.f;
    for (int r = 0; r < R; ++r) a += red[r * mine + tid];
    from_f32(o[bh * dv + first + tid], a);
  }
}

// ---- host -----------------------------------------------------------------------------------------------

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

swimba_status check_la(const swimba_linattn_dims* d) {
  if (d == nullptr || d->batch <= 0 || d->seqlen <= 0 || d->n_heads <= 0 || d->n_kv_heads <= 0 || d->d_k <= 0 ||
      d->d_v <= 0)
    return SWIMBA_ERR_INVALID_ARG;
  if (d->io_dtype != SWIMBA_F32 && d->io_dtype != SWIMBA_BF16) return SWIMBA_ERR_INVALID_ARG;
  if (d->n_heads % d->n_kv_heads != 0) return SWIMBA_ERR_INVALID_ARG;
  if (d->d_k % 8 || d->d_v % 8 || d->d_k > 128 || d->d_v > 128) return SWIMBA_ERR_UNSUPPORTED;
  if (d->n_heads > (1 << 16) || d->batch > (1 << 20) || d->seqlen > (int64_t(1) << 30) ||
      d->batch * d->n_heads > (1 << 22) || d->batch * d->seqlen > (int64_t(1) << 31))
    return SWIMBA_ERR_UNSUPPORTED;
  const int64_t w[3] = {(int64_t)d->n_heads * d->d_k, (int64_t)d->n_kv_heads * d->d_k, (int64_t)d->n_kv_heads * d->d_v};
  const int64_t st[3] = {d->q_stride, d->k_stride, d->v_stride};
  for (int i = 0; i < 3; ++i) {
    if (st[i] < w[i]) return SWIMBA_ERR_INVALID_ARG;
    if (st[i] % 8 || st[i] > (int64_t(1) << 31) || d->seqlen * st[i] > (int64_t(1) << 38)) return SWIMBA_ERR_UNSUPPORTED;
  }
  return SWIMBA_OK;
}

// The tensor-core kernel takes roles of one padded size (64 or 128) together: all three where d_k and
// d_v pad alike, else dq and dk, then dv.
bool la_one_launch(int roles, int d_k, int d_v) { return roles < 3 || (d_k <= 64) == (d_v <= 64); }

// Segments per sequence. Splitting a sequence costs a second pass over y and w (the segments' end
// states), so it pays only where the heads alone leave SMs idle. The rule takes the split with the
// least time in units of one chunk's outputs on one CTA, summed over the launches: rounds of CTAs x chunks per
// segment, with `pass` units more per chunk for the state pass of a split sequence, `state` per segment for its
// state's way through memory and `launch` for the launches more. Tensor cores (a unit is about 3 us):
// 16 heads x 65536 tokens take 0.39 ms in 9 segments, 2.1 ms whole. fp32 (32 tokens, 8 us): 48 roles x
// 333 tokens take 76 us in segments, 176 us whole. Gradients in two launches, heads of 64 x 128, 4096 tokens:
// 24 heads take 138 us in 6 segments, 32 heads 165 in 4 and 192 whole, 40 heads 208 in 3 and 194 whole.
// Whole sequences of as many heads as CTAs or more are dealt out in equal shares where that is less (see run_la_tc),
// unless they have lengths of their own: 160 heads of 128 x 16384 tokens take 0.59 ms so, 1.04 ms in 8 segments.
LaPlan la_plan(const swimba_linattn_dims* d, int roles, bool tc, bool lens) {
  const int chunk = tc ? kLaChunk : kLaSimtChunk;
  const int64_t nch = (d->seqlen + chunk - 1) / chunk;
  const int64_t heads = d->batch * d->n_heads * (tc ? 1 : (std::max(d->d_k, d->d_v) + kSimtCols - 1) / kSimtCols);
  const int64_t slots = tc ? kSMs : 4 * kSMs;
  const bool one = !tc || la_one_launch(roles, d->d_k, d->d_v);
  const double pass = tc ? 0.5 : 0.7, state = tc ? 2 : 0.3, launch = !tc ? 0.7 : one ? 4 : 13;
  const bool cut = tc && !lens && heads * (one ? roles : 2) >= kSMs;
  auto units = [&](int64_t items, int64_t segs, int64_t cps) {
    const double whole = (double)((items * segs + slots - 1) / slots);
    if (segs > 1) return whole * (cps * (1 + pass) + state);
    return cut && items >= kSMs ? std::min(whole * cps, la_shared_units(items * cps, kSMs)) : whole * cps;
  };
  auto time = [&](int64_t segs, int64_t cps) {
    const double t = one ? units(heads * roles, segs, cps) : units(heads * 2, segs, cps) + units(heads, segs, cps);
    return segs > 1 ? t + launch : t;
  };
  LaPlan best{tc, 1, (int)nch, cut};
  double least = time(1, nch);
  for (int64_t n = 2; n <= std::min<int64_t>(nch, 64); ++n) {
    const int64_t cps = (nch + n - 1) / n, segs = (nch + cps - 1) / cps;
    const double t = time(segs, cps);
    if (t < least) {
      least = t;
      best = LaPlan{tc, (int)segs, (int)cps, false};
    }
  }
  return best;
}

struct LaLayout {
  size_t seg[kLaMaxRoles], part_k, part_v, flags, states, total;
};

// bf16 sequences of a few tokens take the recurrence too: a chunk costs the same however few it holds, and nothing
// but the output is rounded. Chunk against recurrence, forward and backward, us of the kernels:
//   64 sequences x 32 heads of 128: 2 tokens 104 / 73 and 257 / 107, 8 tokens 105 / 100 and 257 / 197, 16 tokens
//   105 / 142 and 259 / 339; 4 x 24 heads of 128: 8 tokens 10.5 / 10.6 and 16 / 11, 16 tokens 10.5 / 14.7 and 16 / 18
//   64 x 32 heads of 64: 8 tokens 95 / 30 and 253 / 65; 4 x 24: 8.4 / 6.3 and 14 / 6.5; 1 x 8: 7.7 / 6.3 and 7.4 / 5.6
// (heads of 64 would gain from it up to 16 tokens and more; heads of 128 lose).
constexpr int kLaShort = 8;
static_assert(kLaShort <= kLaSimtChunk, "bf16 sequences on the SIMT cores have one segment");
bool la_use_tc(const swimba_linattn_dims* d) { return d->io_dtype == SWIMBA_BF16 && d->seqlen > kLaShort; }

LaLayout la_layout(const swimba_linattn_dims* d, const LaPlan& pl, int roles) {
  LaLayout l{};
  size_t off = kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  for (int i = 0; i < roles; ++i)
    l.seg[i] = pl.nseg > 1 ? take((size_t)d->batch * d->n_heads * pl.nseg * d->d_k * d->d_v * 4) : 0;
  if (roles > 1 && d->n_kv_heads < d->n_heads) {
    l.part_k = take((size_t)d->batch * d->seqlen * d->n_heads * d->d_k * 4);
    l.part_v = take((size_t)d->batch * d->seqlen * d->n_heads * d->d_v * 4);
  }
  if (pl.cut) {
    l.flags = take(kLaFlagBytes);
    l.states = take(kLaHandBytes);
  }
  l.total = off;
  return l;
}

void launch_chain(const LaParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.n_roles * p.B * p.H), 32);  // 32 x 128 threads: up to 128 x 128 elements
  la_chain_kernel<<<grid, 128, 0, s>>>(p);
  note_launch();
}

template <typename IO, int NI>
cudaError_t launch_simt(const LaParams& p, int max_dw, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.n_roles * p.B * p.H * p.nseg), (unsigned)((max_dw + kSimtCols - 1) / kSimtCols));
  if (p.nseg > 1) {
    if constexpr (sizeof(IO) == 4) la_simt_kernel<IO, NI, 1><<<grid, 128, 0, s>>>(p);
    else return cudaErrorInvalidConfiguration;  // see kLaShort
    note_launch();
    launch_chain(p, s);
  }
  la_simt_kernel<IO, NI, 0><<<grid, 128, 0, s>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <typename IO>
cudaError_t run_simt(const LaParams& p, cudaStream_t s) {
  int dx = 0, dw = 0;
  for (int i = 0; i < p.n_roles; ++i) {
    dx = std::max(dx, p.role[i].dx);
    dw = std::max(dw, p.role[i].dw);
  }
  if (dx <= 32) return launch_simt<IO, 2>(p, dw, s);
  if (dx <= 64) return launch_simt<IO, 4>(p, dw, s);
  return dx <= 96 ? launch_simt<IO, 6>(p, dw, s) : launch_simt<IO, 8>(p, dw, s);
}

cudaError_t run_tc(const LaParams& p, cudaStream_t s) {
  const bool same = la_one_launch(p.n_roles, p.role[0].dx, p.role[0].dw);
  LaParams part[2] = {p, p};
  if (!same) {
    part[0].n_roles = 2;
    part[1].n_roles = 1;
    part[1].role[0] = p.role[2];
  }
  if (p.nseg > 1) {
    for (int i = 0; i < (same ? 1 : 2); ++i) {
      const cudaError_t e = run_la_tc(part[i], true, s);
      if (e != cudaSuccess) return e;
    }
    launch_chain(p, s);
  }
  for (int i = 0; i < (same ? 1 : 2); ++i) {
    const cudaError_t e = run_la_tc(part[i], false, s);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

cudaError_t run_roles(const LaParams& p, bool tc, bool bf16, cudaStream_t s) {
  return tc ? run_tc(p, s) : bf16 ? run_simt<__nv_bfloat16>(p, s) : run_simt<float>(p, s);
}

// One launch over n gradients, whose widest has `width` channels.
void launch_rows(const LaRows& p, int n, int width, bool bf16, cudaStream_t s) {
  if (n == 0) return;
  const dim3 grid((unsigned)((p.B * p.L * (width / 8) + 255) / 256), (unsigned)n);
  if (bf16) la_rows_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
  else la_rows_kernel<float><<<grid, 256, 0, s>>>(p);
  note_launch();
}

float* at(void* ws, size_t off) { return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + off); }

LaParams la_params(const swimba_linattn_dims* d, const LaPlan& pl, const LaLayout& l, const float* g,
                   const int32_t* lens, void* ws) {
  LaParams p{};
  p.hand_flags = pl.cut ? reinterpret_cast<int*>(at(ws, l.flags)) : nullptr;
  p.hand_states = pl.cut ? at(ws, l.states) : nullptr;
  p.g = g;
  p.lens = lens;
  p.L = d->seqlen;
  p.B = (int)d->batch;
  p.H = d->n_heads;
  p.chunk = pl.tc ? kLaChunk : kLaSimtChunk;
  p.nseg = pl.nseg;
  p.cps = pl.cps;
  p.status = ws;
  return p;
}

LaStream la_stream(const void* p, int64_t stride, int64_t L, int div) { return LaStream{p, stride, stride * L, div}; }

}  // namespace
}  // namespace swimba

using namespace swimba;

extern "C" {

size_t swimba_linattn_workspace_size(const swimba_linattn_dims* dims, int op) {
  if (check_la(dims) != SWIMBA_OK || (op != SWIMBA_OP_LINATTN_FWD && op != SWIMBA_OP_LINATTN_BWD)) return 0;
  const int roles = op == SWIMBA_OP_LINATTN_FWD ? 1 : 3;
  const bool tc = la_use_tc(dims);  // enough for a call with lens and for one without
  return std::max(la_layout(dims, la_plan(dims, roles, tc, true), roles).total,
                  la_layout(dims, la_plan(dims, roles, tc, false), roles).total);
}

swimba_status swimba_linattn_fwd(const swimba_linattn_dims* dims, const void* q, const void* k, const void* v,
                                 const float* log_decay, const int32_t* lens, const float* S0, void* o, float* S_final,
                                 void* ws, size_t ws_bytes, void* stream) {
  const swimba_status st = check_la(dims);
  if (st != SWIMBA_OK) return st;
  if (!q || !k || !v || !log_decay || !o || o == q || o == k || o == v) return SWIMBA_ERR_INVALID_ARG;
  const LaPlan pl = la_plan(dims, 1, la_use_tc(dims), lens != nullptr);
  const LaLayout l = la_layout(dims, pl, 1);
  if (ws == nullptr || ws_bytes < l.total) return SWIMBA_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(S0) || !aligned16(S_final) ||
      !aligned16(ws))
    return SWIMBA_ERR_ALIGN;
  LaParams p = la_params(dims, pl, l, log_decay, lens, ws);
  const int group = dims->n_heads / dims->n_kv_heads;
  const int64_t L = dims->seqlen, ow = (int64_t)dims->n_heads * dims->d_v;
  p.n_roles = 1;
  LaRole& r = p.role[0];
  r.x = la_stream(q, dims->q_stride, L, 1);
  r.y = la_stream(k, dims->k_stride, L, group);
  r.w = la_stream(v, dims->v_stride, L, group);
  r.out = o;
  r.out_st = ow;
  r.out_sb = ow * L;
  r.dx = dims->d_k;
  r.dw = dims->d_v;
  r.s_inter = dims->scale;
  r.s_u = 1.f;
  r.M0 = S0;
  r.M_end = S_final;
  r.sj = dims->d_v;
  r.sc = 1;
  r.seg = pl.nseg > 1 ? at(ws, l.seg[0]) : nullptr;
  r.parts = S_final != nullptr ? 3 : 2;
  return api_cuda_status(run_roles(p, pl.tc, dims->io_dtype == SWIMBA_BF16, static_cast<cudaStream_t>(stream)));
}

swimba_status swimba_linattn_step(const swimba_linattn_dims* dims, const void* q, const void* k, const void* v,
                                  const float* log_decay, const float* S_in, void* o, float* S_out, void* stream) {
  const swimba_status st = check_la(dims);
  if (st != SWIMBA_OK) return st;
  if (dims->seqlen != 1 || !q || !k || !v || !log_decay || !S_in || !o || !S_out || o == q || o == k || o == v)
    return SWIMBA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(S_in) || !aligned16(S_out))
    return SWIMBA_ERR_ALIGN;
  const int group = dims->n_heads / dims->n_kv_heads;
  const LaStream sq = la_stream(q, dims->q_stride, 1, 1), sk = la_stream(k, dims->k_stride, 1, group),
                 sv = la_stream(v, dims->v_stride, 1, group);
  const int64_t heads = dims->batch * dims->n_heads;
  const int cols = heads < 2 * kSMs ? 32 : 128;
  const dim3 grid((unsigned)heads, (unsigned)((dims->d_v + cols - 1) / cols));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->io_dtype == SWIMBA_BF16)
    la_step_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(sq, sk, sv, log_decay, S_in, static_cast<__nv_bfloat16*>(o),
                                                      S_out, dims->n_heads, dims->d_k, dims->d_v, cols, dims->scale);
  else
    la_step_kernel<float><<<grid, 256, 0, s>>>(sq, sk, sv, log_decay, S_in, static_cast<float*>(o), S_out,
                                               dims->n_heads, dims->d_k, dims->d_v, cols, dims->scale);
  note_launch();
  return api_cuda_status(cudaGetLastError());
}

swimba_status swimba_linattn_bwd(const swimba_linattn_dims* dims, const void* q, const void* k, const void* v,
                                 const float* log_decay, const int32_t* lens, const float* S0, const void* g_o,
                                 const float* g_S, void* dq, void* dk, void* dv, float* dS0, void* ws, size_t ws_bytes,
                                 void* stream) {
  const swimba_status st = check_la(dims);
  if (st != SWIMBA_OK) return st;
  if (!q || !k || !v || !log_decay || !g_o || !dq || !dk || !dv) return SWIMBA_ERR_INVALID_ARG;
  if (dS0 != nullptr && (dS0 == g_S || dS0 == S0)) return SWIMBA_ERR_INVALID_ARG;  // another role may still read them
  const void* const in[4] = {q, k, v, g_o};
  void* const out[3] = {dq, dk, dv};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 4; ++j)
      if (out[i] == in[j]) return SWIMBA_ERR_INVALID_ARG;
    if (out[i] == out[(i + 1) % 3]) return SWIMBA_ERR_INVALID_ARG;
  }
  const LaPlan pl = la_plan(dims, 3, la_use_tc(dims), lens != nullptr);
  const LaLayout l = la_layout(dims, pl, 3);
  if (ws == nullptr || ws_bytes < l.total) return SWIMBA_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g_o) || !aligned16(dq) || !aligned16(dk) ||
      !aligned16(dv) || !aligned16(S0) || !aligned16(g_S) || !aligned16(dS0) || !aligned16(ws))
    return SWIMBA_ERR_ALIGN;
  LaParams p = la_params(dims, pl, l, log_decay, lens, ws);
  const int H = dims->n_heads, group = H / dims->n_kv_heads, d_k = dims->d_k, d_v = dims->d_v;
  const int64_t L = dims->seqlen, ow = (int64_t)H * d_v;
  const LaStream sq = la_stream(q, dims->q_stride, L, 1), sk = la_stream(k, dims->k_stride, L, group),
                 sv = la_stream(v, dims->v_stride, L, group), sd = la_stream(g_o, ow, L, 1);
  const bool shared = group > 1;
  p.n_roles = 3;
  for (int i = 0; i < 3; ++i) {  // dq, dk, dv (the roles of linattn.cuh)
    LaRole& r = p.role[i];
    r.x = i == 0 ? sd : i == 1 ? sv : sk;
    r.y = i == 0 ? sv : i == 1 ? sd : sq;
    r.w = i == 0 ? sk : i == 1 ? sq : sd;
    r.dx = i == 2 ? d_k : d_v;
    r.dw = i == 2 ? d_v : d_k;
    r.rev = i != 0;
    r.s_inter = i == 0 ? dims->scale : 1.f;
    r.s_u = i == 0 ? 1.f : dims->scale;
    r.M0 = i == 0 ? S0 : g_S;
    r.M_end = i == 2 ? dS0 : nullptr;
    r.sj = i == 2 ? d_v : 1;
    r.sc = i == 2 ? 1 : d_v;
    r.seg = pl.nseg > 1 ? at(ws, l.seg[i]) : nullptr;
    r.parts = r.M_end != nullptr ? 3 : 2;
    if (i > 0 && shared) {
      r.out = at(ws, i == 1 ? l.part_k : l.part_v);
      r.out_st = (int64_t)H * r.dw;
      r.out_f32 = 1;
    } else {
      r.out = out[i];
      r.out_st = i == 0 ? dims->q_stride : i == 1 ? dims->k_stride : dims->v_stride;
    }
    r.out_sb = r.out_st * L;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dims->io_dtype == SWIMBA_BF16;
  const cudaError_t e = run_roles(p, pl.tc, bf16, s);
  if (e != cudaSuccess) return api_cuda_status(e);
  LaRows rows{};
  rows.lens = lens;
  rows.B = dims->batch;
  rows.L = L;
  rows.group = group;
  int n = 0, width = 0;
  auto add = [&](void* dst, int64_t stride, const float* part, int heads, int d) {
    if (part == nullptr && lens == nullptr) return;
    rows.of[n++] = LaRowsOf{dst, stride, part, heads, d};
    width = std::max(width, heads * d);
  };
  add(dq, dims->q_stride, nullptr, H, d_k);
  add(dk, dims->k_stride, shared ? at(ws, l.part_k) : nullptr, dims->n_kv_heads, d_k);
  add(dv, dims->v_stride, shared ? at(ws, l.part_v) : nullptr, dims->n_kv_heads, d_v);
  launch_rows(rows, n, width, bf16, s);
  return api_cuda_status(cudaGetLastError());
}

}  // extern "C"
