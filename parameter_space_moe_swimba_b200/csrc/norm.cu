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
// Bound by memory: every tensor is read or written once, 16 bytes per thread and access. A row belongs to
// one warp (up to 256 channels) or one CTA of up to 512 threads, which walks its rows with the next ones
// on their way: each thread copies the vectors of 8 channels that it will work on into shared memory of
// its own (cp.async, no barrier), as many rows ahead as fit, and keeps its channels' weights and their gradients in
// registers. (Above 8192 channels a thread has 32, and the backward's 128 registers do not hold them: 1.2 KB of them
// and of the row's values per thread go to local memory; 2048 rows of 16384 in bf16 take 316 to 425 us for 82 of
// bytes, in fp32 500 for 164.) Without the copies a row's loads waited for the row before it (16384 rows of 4096, bf16
// with an fp32 residual, backward: 547 us, 2.7 TB/s); with 8 channels per thread a third of the
// instructions were the row's sums and addresses, so a thread takes 16 where rows are long. Now that backward
// takes 389 us (3.8 TB/s, 58 % of the measured copy rate: 1300 instructions per warp and row at 40 % of the
// issue slots, the row's three sums and the copies' shared memory the rest, with two CTAs of 8 warps on an SM,
// as the registers allow), the forward of 32768 rows of 4096 in bf16 228 us (90 %).
// All sums are fp32 and taken in a fixed order.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "sm100.cuh"

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

// Two floats in one 64-bit register pair: the packed fp32 instructions round each as the scalar ones do and
// take half the issue slots, which bound the backward (439 -> 400 us; the forward, which memory bounds, is
// faster with scalar ones: 240 against 267 us).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 f2_split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// 1 / (1 + e^-z) with the exp2 and reciprocal instructions (each within 2^-22).
__device__ __forceinline__ float f_sigmoid(float z) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(-kLog2e * z)));
  return r;
}
__device__ __forceinline__ F2 f2_sigmoid(F2 z) {
  const float2 t = f2_split(z * f2(-kLog2e));
  const float2 d = f2_split(f2(ex2_approx(t.x), ex2_approx(t.y)) + f2(1.f));
  float a, b;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(d.y));
  return f2(a, b);
}
template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, const F2 (&v)[4]) {
  T* p = reinterpret_cast<T*>(base) + at;
  const float2 a = f2_split(v[0]), b = f2_split(v[1]), c = f2_split(v[2]), d = f2_split(v[3]);
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(a.x, a.y), bf16x2(b.x, b.y), bf16x2(c.x, c.y), bf16x2(d.x, d.y));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
  }
}

// A row's threads: one warp of a CTA of four (WARP), or a whole CTA.
template <bool WARP>
__device__ __forceinline__ void row_sync() {
  if constexpr (WARP) __syncwarp();
  else __syncthreads();
}

// Sums of K values over the threads of a row, the same in every thread. `red`: 16 K floats of shared
// memory that no other sum of this row uses between two row_syncs.
template <bool WARP, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (!WARP) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[k * 16 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = lane < warps ? red[k * 16 + lane] : 0.f;
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      v[k] = __shfl_sync(0xffffffffu, s, 0);
      if (warps > 8) v[k] += __shfl_sync(0xffffffffu, s, 8);
    }
  }
}

// Sums over the groups of a row: v[i] is this thread's sum over its vector i (tid + i tpr), and becomes the
// sum over the group that the vector lies in. Groups of 8, 16 .. 256 channels in powers of two are whole
// aligned sets of lanes and meet in shuffles; others go through shared memory (`gred`: a float per
// vector and one per group), one warp per group.
template <bool WARP, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], int nvec, int groups, int tid, int tpr, float* red, float* gred) {
  if (groups == 1) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) s[0] += v[i];
    row_sum<WARP, 1>(s, red);
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
    if (tid + i * tpr < nvec) gred[tid + i * tpr] = v[i];
  row_sync<WARP>();
  const int lane = tid & 31;
  for (int g = tid >> 5; g < groups; g += tpr >> 5) {
    float s = 0.f;
    for (int j = lane; j < gv; j += 32) s += gred[g * gv + j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) gsum[g] = s;
  }
  row_sync<WARP>();
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + i * tpr < nvec) v[i] = gsum[(tid + i * tpr) / gv];
}

constexpr int kRed = 64;     // floats of row_sum's shared memory: 16 + 32 + 16; two sets, for even and odd rows
constexpr int kInputs = 5;   // y, z, res, g_h, g_n

// The row inputs: read from the thread's own copies in shared memory, which hold STAGES rows (one at work,
// the others on their way), or, with STAGES = 0, from global memory. STAGES = 1 (backward) is where two
// whole rows do not fit: y and z, which a row needs to its end, have two places, and res, g_h and g_n, which
// it has done with in its middle, one each, filled for the next row from there on (2048 rows of 16384 in bf16:
// 406 us from global memory, 316 so; 8192 of 4096 in fp32: 321 us with one place of each, 306 so).
// Neighbouring threads' pieces lie side by side: with a thread's pieces together, at an odd pitch, the copies
// took as long again (forward 223 -> 355 us).
template <typename IO, typename RES, int NV, int STAGES>
struct RowInputs {
  const void* src[kInputs];
  uint32_t at[kInputs];  // of the tensor's part of a stage, this thread's first 16 bytes
  uint32_t stage, bytes;  // the row at work's place, and the distance between two
  static constexpr bool kSplit = STAGES == 1;
  static constexpr int kPlaces = kSplit ? 2 : STAGES, kTwice = 2;  // inputs before kTwice have two places
  int nvec, tid, tpr, width;
  int64_t row;

  static constexpr bool kRes(int k) { return k == 2 || k == 3; }
  static constexpr int kParts(int k) { return (kRes(k) ? sizeof(RES) : sizeof(IO)) == 4 ? 2 : 1; }

  __device__ __forceinline__ RowInputs(const NormParams& p, uint32_t smem, int tid_, int tpr_)
      : src{p.y, p.z, p.res, p.g_h, p.g_n}, nvec(p.width / 8), tid(tid_), tpr(tpr_), width(p.width), row(0) {
    uint32_t off = 0;
#pragma unroll
    for (int k = 0; k < kInputs; ++k) {
      at[k] = smem + off + tid * 16;
      if (src[k]) off += NV * tpr * 16 * kParts(k);
      if (kSplit && k == kTwice - 1) bytes = off, off *= 2;
    }
    stage = 0;
    if (!kSplit) bytes = off;
  }
  // Starts this thread's copies of inputs FROM to TO - 1 of row r into a place (an empty group behind the
  // last row). `ahead` is the row's distance in channels from the tensors' beginnings.
  template <int FROM = 0, int TO = kSplit ? kTwice : kInputs>
  __device__ __forceinline__ void fetch(int64_t r, int64_t rows, int64_t ahead, uint32_t st) {
    if constexpr (STAGES == 0) return;
    if (r < rows) {
#pragma unroll
      for (int k = FROM; k < TO; ++k) {
        if (!src[k]) continue;
        const uint8_t* from = reinterpret_cast<const uint8_t*>(src[k]) + ahead * (kParts(k) * 2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = tid + i * tpr;
          if (v >= nvec) continue;
#pragma unroll
          for (int h = 0; h < kParts(k); ++h)
            sm100::cp_async16(at[k] + st * bytes + (h * NV + i) * tpr * 16, from + v * (16 * kParts(k)) + h * 16);
        }
      }
    }
    sm100::cp_async_commit();
  }
  __device__ __forceinline__ void use(int64_t r, uint32_t st) {
    row = r;
    stage = st * bytes;
    if constexpr (STAGES > 0) sm100::cp_async_wait<kSplit ? 2 : STAGES - 1>();
  }
  // kSplit's groups are y and z of a row, then the rest of it, then y and z of the next.
  __device__ __forceinline__ void fetch_rest(int64_t r, int64_t rows, int64_t ahead) {
    if constexpr (kSplit) fetch<kTwice, kInputs>(r, rows, ahead, 0);
  }
  __device__ __forceinline__ void use_rest() {
    if constexpr (kSplit) sm100::cp_async_wait<1>();
  }
  template <int K>
  __device__ __forceinline__ void get(int i, float (&v)[8]) const {
    using T = typename std::conditional<kRes(K), RES, IO>::type;
    if constexpr (STAGES == 0) {
      load8<T>(src[K], row * width + 8 * (tid + i * tpr), v);
    } else {
      auto part = [&](int h) {
        uint4 q;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "r"(at[K] + (kSplit && K >= kTwice ? 0 : stage) + (h * NV + i) * tpr * 16));
        return q;
      };
      if constexpr (sizeof(T) == 2) {
        Vec16<__nv_bfloat16>::unpack(part(0), v);
      } else {
        const uint4 a = part(0), b = part(1);
        v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
      }
    }
  }
  template <int K>
  __device__ __forceinline__ void get(int i, F2 (&v)[4]) const {
    float f[8];
    get<K>(i, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f2(f[2 * e], f[2 * e + 1]);
  }
};

// Shared memory of a row's threads: the cross-warp sums and, for groups that need it, group_sum's (both
// rounded to 16 bytes), then the stages.
__host__ __device__ inline bool norm_groups_in_smem(int nvec, int groups) {
  const int gv = nvec / groups;
  return groups > 1 && (gv > 32 || (gv & (gv - 1)) != 0);
}
__host__ __device__ inline int norm_sum_floats(int nvec, int groups) {
  return (2 * kRed + (norm_groups_in_smem(nvec, groups) ? nvec + groups : 0) + 3) & ~3;
}

template <bool WARP>
struct RowThreads {
  int tid, tpr, slot, per_cta;
  __device__ __forceinline__ RowThreads()
      : tid(WARP ? threadIdx.x & 31 : threadIdx.x), tpr(WARP ? 32 : blockDim.x), slot(WARP ? threadIdx.x >> 5 : 0),
        per_cta(WARP ? blockDim.x >> 5 : 1) {}
};

// ---- forward ---------------------------------------------------------------------------------------------
template <typename IO, typename RES, int NV, bool WARP, int STAGES, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1) norm_fwd_kernel(const NormParams p, int slot_bytes) {
  extern __shared__ __align__(16) float smem[];
  const RowThreads<WARP> t;
  const int tid = t.tid, tpr = t.tpr, nvec = p.width / 8;
  float* red = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(smem) + t.slot * slot_bytes);
  float* gred = red + 2 * kRed;
  const bool group_smem = norm_groups_in_smem(nvec, p.groups);
  RowInputs<IO, RES, NV, STAGES> in(p, sm100::smem_u32(red + norm_sum_floats(nvec, p.groups)), tid, tpr);
  const int64_t first = (int64_t)blockIdx.x * t.per_cta + t.slot, step = (int64_t)gridDim.x * t.per_cta;
  const float inv = 1.f / (float)p.width, ginv = (float)p.groups / (float)p.width;
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) in.fetch(first + k * step, p.rows, (first + k * step) * p.width, k);
  float wp[NV][8], wn[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * tpr;
    if (v >= nvec) continue;
    if (p.w_post) load8<float>(p.w_post, 8 * v, wp[i]);
    if (p.w_pre) load8<float>(p.w_pre, 8 * v, wn[i]);
  }
  uint32_t st = 0;
  int red_row = 0;
  for (int64_t row = first; row < p.rows; row += step) {
    const int64_t next = row + (STAGES - 1) * step;
    in.fetch(next, p.rows, next * p.width, st == 0 ? STAGES - 1 : st - 1);
    in.use(row, st);
    if (++st == STAGES) st = 0;
    float a[NV][8];
    float s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i][e] = 0.f;
      if (tid + i * tpr >= nvec) continue;
      if (p.y) in.template get<0>(i, a[i]);
      if (p.z && !p.gate_last) {
        float z[8];
        in.template get<1>(i, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] *= z[e] * f_sigmoid(z[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i] = fmaf(a[i][e], a[i][e], s[i]);
    }
    if (p.w_post) {
      group_sum<WARP, NV>(s, nvec, p.groups, tid, tpr, red + red_row, gred);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float r = rsqrtf(fmaf(s[i], ginv, p.eps)) * p.beta;
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] *= r * wp[i][e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] *= p.beta;
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * tpr;
      if (v >= nvec) continue;
      if (p.z && p.gate_last) {
        float z[8];
        in.template get<1>(i, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] *= z[e] * f_sigmoid(z[e]);
      }
      float r[8];
      if (p.res) in.template get<2>(i, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (p.res) a[i][e] = fmaf(p.alpha, r[e], a[i][e]);
        ss[0] = fmaf(a[i][e], a[i][e], ss[0]);
      }
      if (p.h) store8<RES>(p.h, row * p.width + 8 * v, a[i]);
    }
    if (p.n) {
      row_sum<WARP, 1>(ss, red + red_row + 16);
      const float r = rsqrtf(fmaf(ss[0], inv, p.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * tpr;
        if (v >= nvec) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] *= r * wn[i][e];
        store8<IO>(p.n, row * p.width + 8 * v, a[i]);
      }
    }
    // the next row's sums go into the other set; group_sum's shared memory has one
    red_row ^= kRed;
    if (group_smem) row_sync<WARP>();
  }
}

// ---- backward --------------------------------------------------------------------------------------------
// A CTA writes its sums of the two weight gradients once, to be summed over the CTAs by norm_dw_kernel.
template <typename IO, typename RES, int NV, bool WARP, int STAGES, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) norm_bwd_kernel(const NormParams p, int slot_bytes) {
  extern __shared__ __align__(16) float smem[];
  const RowThreads<WARP> t;
  const int tid = t.tid, tpr = t.tpr, nvec = p.width / 8;
  float* red = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(smem) + t.slot * slot_bytes);
  float* gred = red + 2 * kRed;
  const bool group_smem = norm_groups_in_smem(nvec, p.groups);
  using In = RowInputs<IO, RES, NV, STAGES>;
  In in(p, sm100::smem_u32(red + norm_sum_floats(nvec, p.groups)), tid, tpr);
  const int64_t first = (int64_t)blockIdx.x * t.per_cta + t.slot, step = (int64_t)gridDim.x * t.per_cta;
  const float inv = 1.f / (float)p.width, ginv = (float)p.groups / (float)p.width;
#pragma unroll
  for (int k = 0; k < In::kPlaces - 1; ++k) in.fetch(first + k * step, p.rows, (first + k * step) * p.width, k);
  in.fetch_rest(first, p.rows, first * p.width);
  F2 wp[NV][4], wn[NV][4], dwp[NV][4], dwn[NV][4];  // wp: β w_post; dwp without its β until the end
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * tpr;
    float a[8] = {}, b[8] = {};
    if (v < nvec && p.w_post) load8<float>(p.w_post, 8 * v, a);
    if (v < nvec && p.w_pre) load8<float>(p.w_pre, 8 * v, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      wp[i][e] = p.w_post ? f2(p.beta * a[2 * e], p.beta * a[2 * e + 1]) : f2(p.beta);
      wn[i][e] = f2(b[2 * e], b[2 * e + 1]);
      dwp[i][e] = dwn[i][e] = f2(0.f);
    }
  }
  const bool gate_first = p.z && !p.gate_last, gate_last = p.z && p.gate_last;
  uint32_t st = 0;
  int red_row = 0;
  int64_t ahead = (first + (In::kPlaces - 1) * step) * p.width;
  for (int64_t row = first; row < p.rows; row += step) {
    in.fetch(row + (In::kPlaces - 1) * step, p.rows, ahead, st == 0 ? In::kPlaces - 1 : st - 1);
    in.use(row, st);
    if (++st == In::kPlaces) st = 0;
    const int64_t base = row * p.width;
    // the forward: a, its norm, h
    F2 hat[NV][4], h[NV][4];
    float r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) hat[i][e] = h[i][e] = f2(0.f);
      if (tid + i * tpr >= nvec) continue;
      if (p.y) in.template get<0>(i, hat[i]);
      if (gate_first) {
        F2 z[4];
        in.template get<1>(i, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) hat[i][e] = hat[i][e] * (z[e] * f2_sigmoid(z[e]));
      }
      F2 q = f2(0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) q = f2_fma(hat[i][e], hat[i][e], q);
      r[i] = f2_split(q).x + f2_split(q).y;
    }
    if (p.w_post) {
      group_sum<WARP, NV>(r, nvec, p.groups, tid, tpr, red + red_row, gred);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        r[i] = rsqrtf(fmaf(r[i], ginv, p.eps));
#pragma unroll
        for (int e = 0; e < 4; ++e) hat[i][e] = hat[i][e] * f2(r[i]);
      }
    }
    in.use_rest();
    float s[2] = {0.f, 0.f};
    if (p.g_n) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (tid + i * tpr >= nvec) continue;
        F2 z[4], gn[4];
        if (gate_last) in.template get<1>(i, z);
        if (p.res) in.template get<2>(i, h[i]);
        in.template get<4>(i, gn);
        F2 s0 = f2(0.f), s1 = f2(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          F2 q = hat[i][e] * wp[i][e];
          if (gate_last) q = q * (z[e] * f2_sigmoid(z[e]));
          h[i][e] = f2_fma(f2(p.alpha), h[i][e], q);
          s0 = f2_fma(h[i][e], h[i][e], s0);
          s1 = f2_fma(gn[e] * wn[i][e], h[i][e], s1);
        }
        s[0] += f2_split(s0).x + f2_split(s0).y;
        s[1] += f2_split(s1).x + f2_split(s1).y;
      }
      row_sum<WARP, 2>(s, red + red_row + 16);
    }
    const float rh = p.g_n ? rsqrtf(fmaf(s[0], inv, p.eps)) : 0.f, back = -(s[1] * rh * inv) * rh * rh;  // (rh³ alone would leave the range first)
    // back through the norm before the next block, the residual, the gate behind the norm
    float q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * tpr;
      q[i] = 0.f;
      if (v >= nvec) continue;
      F2 dh[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
      if (p.g_h) in.template get<3>(i, dh);
      if (p.g_n) {
        F2 gn[4];
        in.template get<4>(i, gn);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 g = gn[e] * f2(rh);
          dwn[i][e] = f2_fma(g, h[i][e], dwn[i][e]);
          dh[e] = f2_fma(h[i][e], f2(back), f2_fma(g, wn[i][e], dh[e]));
        }
      }
      if (p.dres) {
        F2 d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = dh[e] * f2(p.alpha);
        store8<RES>(p.dres, base + 8 * v, d);
      }
      if (gate_last) {
        F2 z[4], dz[4];
        in.template get<1>(i, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 sg = f2_sigmoid(z[e]), zs = z[e] * sg;
          dz[e] = dh[e] * (hat[i][e] * wp[i][e]) * f2_fma(zs, f2_fma(sg, f2(-1.f), f2(1.f)), sg);
          dh[e] = dh[e] * zs;
        }
        store8<IO>(p.dz, base + 8 * v, dz);
      }
      F2 qq = f2(0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dwp[i][e] = f2_fma(dh[e], hat[i][e], dwp[i][e]);
        h[i][e] = dh[e] * wp[i][e];
        qq = f2_fma(h[i][e], hat[i][e], qq);
      }
      q[i] = f2_split(qq).x + f2_split(qq).y;
    }
    in.fetch_rest(row + step, p.rows, ahead);
    ahead += step * p.width;
    // the norm after the mixer and the gate before it
    if (p.w_post) group_sum<WARP, NV>(q, nvec, p.groups, tid, tpr, red + red_row + 48, gred);
    if (p.y) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * tpr;
        if (v >= nvec) continue;
        if (p.w_post) {
          const float mq = -q[i] * ginv;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[i][e] = f2(r[i]) * f2_fma(hat[i][e], f2(mq), h[i][e]);
        }
        if (gate_first) {
          F2 y[4], z[4], dz[4];
          in.template get<0>(i, y);
          in.template get<1>(i, z);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const F2 sg = f2_sigmoid(z[e]), zs = z[e] * sg;
            dz[e] = h[i][e] * y[e] * f2_fma(zs, f2_fma(sg, f2(-1.f), f2(1.f)), sg);
            h[i][e] = h[i][e] * zs;
          }
          store8<IO>(p.dz, base + 8 * v, dz);
        }
        store8<IO>(p.dy, base + 8 * v, h[i]);
      }
    }
    // the next row's sums go into the other set; group_sum's shared memory has one
    red_row ^= kRed;
    if (group_smem) row_sync<WARP>();
  }
  pdl_trigger();
  if (p.part == nullptr) return;
  // this CTA's sums; a CTA's warps with a row each add up one after the other
  float* part = p.part + (size_t)blockIdx.x * 2 * p.width;
  for (int k = 0; k < t.per_cta; ++k) {
    if (k == t.slot) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * tpr;
        if (v >= nvec) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float* d = part + (size_t)w * p.width + 8 * v;
          F2 o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[e] = w ? dwn[i][e] : dwp[i][e] * f2(p.beta);
            if (k > 0) o[e] = o[e] + f2(d[2 * e], d[2 * e + 1]);
          }
          store8<float>(d, 0, o);
        }
      }
    }
    if (WARP) __syncthreads();
  }
}

// dw[c] = Σ over CTAs of part[cta][which][c]: 32 threads per column, each every 32nd CTA.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int ctas, int width, float* dw_post, float* dw_pre) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5, which = blockIdx.y;
  float* out = which ? dw_pre : dw_post;
  pdl_wait();
  float s = 0.f;
  if (out != nullptr && c < width) {
#pragma unroll 4
    for (int i = k; i < ctas; i += 32) s += part[((size_t)i * 2 + which) * width + c];
  }
  red[k][threadIdx.x & 31] = s;
  __syncthreads();
  s = red[threadIdx.x & 31][k];  // warp k: the 32 sums of column k
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0 && out != nullptr && blockIdx.x * 32 + k < width) out[blockIdx.x * 32 + k] = s;
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

// How a call runs: threads per CTA, rows that a CTA works on at a time, CTAs, shared memory per row at work,
// vectors of 8 channels per thread, rows in shared memory.
struct NormPlan {
  int threads, per_cta, ctas, slot_bytes, nv, stages;
  bool warp;
};

NormPlan norm_plan(const swimba_norm_dims* d, bool bwd) {
  NormPlan n{};
  const int nvec = d->width / 8;
  // One vector per thread up to 1024 channels (backward: 2048), two up to 8192, four up to 16384, in whole
  // warps. Two cost fewer instructions, one leaves the backward more warps: at 32768 rows of 1536 the
  // forward takes 91 us with two and 117 with one, the backward 269 and 240.
  n.nv = nvec <= (bwd ? 256 : 128) ? 1 : nvec <= 1024 ? 2 : 4;
  n.warp = nvec <= 32;
  const int tpr = n.warp ? 32 : ((nvec + n.nv - 1) / n.nv + 31) / 32 * 32;
  n.threads = n.warp ? 128 : tpr;
  n.per_cta = n.warp ? 4 : 1;
  // as many rows in shared memory, up to three, as fit (as if every input were given) where a CTA has
  // up to 256 threads beside another one (113 KB each), else alone (226 KB); where only one does, the
  // backward keeps y and z of two and the rest of one
  const size_t io = d->io_dtype == SWIMBA_BF16 ? 2 : 4, res = d->res_dtype == SWIMBA_BF16 ? 2 : 4;
  const size_t sums = (size_t)norm_sum_floats(nvec, d->groups) * 4;
  const size_t stage = (size_t)n.nv * tpr * 8 * (bwd ? 3 * io + 2 * res : 2 * io + res);
  const size_t pair = 113 * 1024, alone = 226 * 1024;
  auto fits = [&](int st, size_t room) { return (sums + st * stage) * n.per_cta <= room; };
  const size_t split = (size_t)n.nv * tpr * 8 * (5 * io + 2 * res);
  if (n.threads <= 256) n.stages = fits(3, pair) ? 3 : fits(2, pair) ? 2 : 1;
  else n.stages = fits(2, alone) ? 2 : bwd && sums + split <= alone ? 1 : 0;
  n.slot_bytes = (int)(sums + (n.stages == 1 ? split : n.stages * stage));
  const int fit = (int)std::min<size_t>(alone / ((size_t)n.slot_bytes * n.per_cta), 16);
  // (the backward's registers allow 512 threads of two vectors, 768 of one); no more CTAs than share the
  // rows evenly, since each writes its partial weight gradients
  const int per_sm = std::max(1, std::min(fit, (bwd ? (n.nv == 1 ? 768 : 512) : 1024) / n.threads));
  const int64_t units = (d->rows + n.per_cta - 1) / n.per_cta, rounds = (units + kSMs * per_sm - 1) / (kSMs * per_sm);
  n.ctas = (int)((units + rounds - 1) / rounds);
  return n;
}

template <typename IO, typename RES, int NV, bool WARP, int STAGES, int MAXT>
cudaError_t launch_norm(const NormPlan& n, const NormParams& p, bool bwd, cudaStream_t s) {
  const int smem = n.slot_bytes * n.per_cta;
  if (n.stages != STAGES || n.nv != NV || n.threads > MAXT) return cudaErrorInvalidConfiguration;
  auto kernel = norm_bwd_kernel<IO, RES, NV, WARP, STAGES, MAXT>;
  if constexpr (STAGES != 1) kernel = bwd ? kernel : norm_fwd_kernel<IO, RES, NV, WARP, STAGES, MAXT>;
  else if (!bwd) return cudaErrorInvalidConfiguration;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)n.ctas, n.threads, smem, s>>>(p, n.slot_bytes);
  note_launch();
  return cudaGetLastError();
}

template <typename IO, typename RES>
cudaError_t run_norm(const swimba_norm_dims* d, const NormParams& p, bool bwd, cudaStream_t s) {
  const NormPlan n = norm_plan(d, bwd);
  // (up to 256 channels three rows always fit, up to 2048 two, up to 4096 two of the forward's)
  if (n.warp) return launch_norm<IO, RES, 1, true, 3, 128>(n, p, bwd, s);
  if (n.nv == 1)
    return n.stages == 3 ? launch_norm<IO, RES, 1, false, 3, 256>(n, p, bwd, s)
                         : launch_norm<IO, RES, 1, false, 2, 256>(n, p, bwd, s);
  if (n.nv == 2 && n.threads <= 256)
    return n.stages == 3   ? launch_norm<IO, RES, 2, false, 3, 256>(n, p, bwd, s)
           : n.stages == 2 ? launch_norm<IO, RES, 2, false, 2, 256>(n, p, bwd, s)
                           : launch_norm<IO, RES, 2, false, 1, 256>(n, p, bwd, s);
  if (n.nv == 2)
    return n.stages == 2   ? launch_norm<IO, RES, 2, false, 2, 512>(n, p, bwd, s)
           : n.stages == 1 ? launch_norm<IO, RES, 2, false, 1, 512>(n, p, bwd, s)
                           : launch_norm<IO, RES, 2, false, 0, 512>(n, p, bwd, s);
  return n.stages == 2   ? launch_norm<IO, RES, 4, false, 2, 512>(n, p, bwd, s)
         : n.stages == 1 ? launch_norm<IO, RES, 4, false, 1, 512>(n, p, bwd, s)
                         : launch_norm<IO, RES, 4, false, 0, 512>(n, p, bwd, s);
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
  return kStatusBytes + (size_t)norm_plan(dims, true).ctas * 2 * dims->width * sizeof(float);
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
  const cudaError_t e2 = launch_pdl(norm_dw_kernel, dim3((unsigned)((dims->width + 31) / 32), 2), dim3(1024), 0, s, p.part,
                                    norm_plan(dims, true).ctas, dims->width, dw_post, dw_pre);
  note_launch();
  return api_cuda_status(e2);
}

}  // extern "C"
