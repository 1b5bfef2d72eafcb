// Linear attention with a decay for each head, in chunks of 128 tokens on the tcgen05 tensor cores
// (bf16 tensors of more than a few tokens; the roles are those of linattn.cuh, in forward order here).
//
// For a chunk of n <= 128 tokens and the state M [dx, dw] before it, with γ = exp(log_decay):
//   P[i, s]  = γ^(i-s) (x_i · y_s) for s <= i, else 0          A = X, B = Y        (K = dx)
//   out_i    = s_intra Σ_s P[i, s] w_s + s_inter γ^(i+1) Mᵀ x_i  A = P, B = W (K = tokens); A = X, B = M
//   M       <- γ^n M + s_u Σ_s y_s γ^(n-1-s) w_sᵀ              A = (γ w)ᵀ, B = Y    (K = tokens)
// A reverse role mirrors the exponents: γ^(s-i) for s >= i, γ^(n-1-i), γ^(s+1).
//
// Persistent, one CTA per SM; an item is one (role, segment, sequence, head), its chunks in order:
//   warp 0       TMA loads of the X, Y, W tiles into a ring each; the item's table of powers of γ; every chunk's γ^n
//   warp 1       the MMAs of scores, readout and outputs
//   warp 2       the MMAs of U. (A wait costs an issuing warp about 170 cycles and a commit 70, as much as
//                two and one of these MMAs, and few MMAs queue up: one warp for both made every wait
//                a gap in the tensor cores' work.)
//   warp 3       TMA stores of the finished output tiles
//   warps 4-11   one row i = TMEM lane each, two warps per row with half of its columns: scores -> P
//                (bf16, in place, the A operand of P W); the carried state's readout scaled in place,
//                to which the MMA adds P W; the sum into the W tile, which no MMA reads any more, and
//                from there to memory
//   warps 12-15  one column c of M each, in fp32 registers for the whole item: M's bf16 copy for the
//                readout (the only rounding of M), M <- γ^n M + U. (U is summed apart from M: the tensor
//                cores' own accumulation would lose a little of M at every step.)
//   warps 16-23  (γ w)ᵀ as two or three bf16 parts into tensor memory (a ring of 16- or 32-token slots, filled
//                by two sets of four warps)
// Except for M's columns all loops stay rolled: six kinds of warps share the instruction cache, whose misses
// go to a cache that the SMs of a cluster share in their turn. With every loop unrolled, a chunk took a
// quarter longer on SMs with 15 neighbours at work than on those with few.
// Where there are as many sequences and heads as CTAs, all chunks are dealt to the CTAs in equal shares:
// a CTA's share then begins and ends inside a sequence. It first does the beginning of the sequence that
// its share ends in and hands the state over in global memory, then its whole sequences, and last the
// rest of the sequence that its share begins in, whose state the CTA before it handed over at its start.
// (256 sequences and heads on 148 CTAs: 56 chunks per CTA in place of 64.)
//
// Rounded to bf16: P and M's copy, once each, because each meets a bf16 operand and makes a bf16
// output; γ w enters M as hi + mid + lo, 24 bits together, where it matters to an fp32 state: where M is
// an output and the chunk's decay to the sequence's end is more than 2^-6; else as hi + mid, 16 bits (all
// through, they would put 3e-6 into S_final and dS0; so they put 1e-7).
// Tensor memory: scores / P 128 columns, out dw, U dx, the γ w ring 96 or 192.
// P's tokens 0-63 lie in columns 0-31, tokens 64-127 in columns 64-95: where the same warp has read scores.
// Bound: a forward of 32 heads of 128 moves 1.09 GB for 8 x 4096 tokens and computes 0.17 TFLOP (P whole, M in
// two parts). It takes 235 us alone (4.6 TB/s and 0.73 PFLOP/s, 71 % and 45 % of the measured peaks) and 264 us
// back to back, where the board's power limit lowers the clock to 1.5 GHz. Heads of 64 are bound by the chain of
// waits inside a chunk; one long sequence reads k and v twice (MODE 1, then MODE 0).
// Every wait is bounded; a wait that runs out records SWIMBA_ERR_TIMEOUT, and the CTA drains and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "linattn.cuh"
#include "sm100.cuh"

namespace swimba {

using namespace sm100;

namespace {

constexpr int kTile = kLaChunk * 128;  // 128 tokens x 128 bytes (64 bf16), 128-byte swizzle: 16 KB
constexpr int kThreads = 768;
// γ w ring: per 16 tokens (one MMA step) 3 parts x 8 columns.
constexpr int kPart = 8, kStep = 16;
constexpr uint32_t kColP = 0, kColO = 128;

// An item's powers of γ by distance, with 32 zeros on the side that the mask hides: 0 .. 0 γ^0 .. γ^127, or
// for a reverse role γ^127 .. γ^0 0 .. 0, so that row i's factor for token s is element la_origin + i - s.
constexpr int kTable = 32 + kLaChunk;
__host__ __device__ constexpr int la_origin(bool rev) { return rev ? kLaChunk - 1 : 32; }

struct LaTcArgs {
  CUtensorMap map[kLaMaxRoles][4];
  LaParams p;
  uint32_t items;
  uint32_t share, extra;  // balanced: chunks per CTA, and how many CTAs have one more
};

enum { kMapX, kMapY, kMapW, kMapOut };

template <int DX, int DW, int MODE>
struct LaSmem {
  static constexpr int XB = DX / 64, WB = DW / 64;
  // The ring's slots are 32 tokens, two MMA steps, each filled by one set of warps: the issuing warp spends
  // about 450 cycles on a slot beside its MMAs, and a set about 500 on a step. Only four slots fit where
  // both sizes are 128; there they are 16 tokens (two of 32 were 2 % slower). Without scores and outputs
  // there is room for two U, and the warps that would make them fill the ring too.
  static constexpr int NU = MODE == 0 ? 1 : 2, RING = 4, SUB = MODE == 0 && DX + DW == 256 ? 1 : 2;
  static constexpr int GROUPS = (MODE == 0 ? 2 : 4) / SUB;  // SUB sets fill a slot, GROUPS slots are filled at a time
  static constexpr int SLOTS = kLaChunk / (kStep * SUB);     // per chunk
  static constexpr uint32_t COL_U = MODE == 0 ? kColO + DW : 0, COL_RING = MODE == 0 ? COL_U + DX : 256;
  static_assert(COL_RING + RING * SUB * 3 * kPart <= 512, "tensor memory");
  static constexpr int TX = MODE == 0 ? XB * kTile : 0, TY = XB * kTile, TW = WB * kTile;  // one tile of each
  static constexpr int COPY = MODE == 0 ? DX * DW * 2 : 0;  // M's bf16 copy, [dw rows][dx], K-major
  // Tiles in flight. An X tile is free after two MMAs, a Y tile after U, a W tile only when the outputs
  // that replace it have left; so W gets the most.
  static constexpr int NX = DX == 128 && DW == 128 ? 1 : 2, NY = DX == 64 ? 3 : 2, NW = DW == 128 ? 3 : 4;
  static constexpr int X = 0, Y = NX * TX, W = Y + NY * TY, M = W + NW * TW;
  static constexpr int POW = M + COPY;              // 2 x kTable floats
  static constexpr int BAR = POW + 2 * kTable * 4;  // barriers
  static constexpr int NBAR = 2 * NX + 2 * NY + 4 * NW + 6 + 2 * RING + 2 * NU + 4 + 2 + 2;
  static constexpr int MISC = BAR + NBAR * 8;
  // γ^n of the chunks in flight. A W tile is loaded where the outputs NW chunks before it (MODE 1: U) are done, so
  // where the state of NW + 1 (NW + 2) chunks before it is: that many factors are in use.
  static constexpr int FACTORS = 8, FACTOR = MISC + 16;
  static_assert(NW + 2 <= FACTORS);
  static constexpr int BYTES = FACTOR + FACTORS * 4;
  // Registers per thread of the six warpgroups (0-3, 4-7 and 8-11, 12-15, 16-19 and 20-23). A spill in one of
  // the chunk loops costs several percent. With DX = 128 (outputs) 18 to 24 words are spilled all the same: given more
  // registers each in turn, two thirds of the stores go with the state's warps, the rest with warps 0-3 and 4-11.
  static constexpr int REG_UTIL = DX == 128 ? 48 : DW == 128 ? 72 : 48, REG_PO = DX == 128 ? 64 : DW == 128 ? 72 : 80,
                       REG_M = DX == 128 ? 176 : DW == 128 ? 120 : 144, REG_W = DX == 128 ? 64 : DW == 128 ? 72 : 64;
  static_assert(REG_UTIL + 2 * REG_PO + REG_M + 2 * REG_W <= 6 * 80, "what the launch's 80 registers per thread allow");
  static_assert(BYTES + 1024 <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ uint32_t swz16(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ uint32_t pair(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Shared memory through its own address space: pointers cut from the aligned base are generic to the
// compiler, and generic accesses cost a chunk several times its arithmetic (8.0 against 0.6 thousand
// cycles for P's 128 x 128 factors).
__device__ __forceinline__ float lds1(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Four 8 x 8 matrices of bf16, transposed: thread t gets of matrix k the elements (2 (t % 4) + 0..1, t / 4)
// of the stored one, whose row i starts at the address that thread 8 k + i gives.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
// 16 lanes x 8 columns: thread t's r[2 k] is lane t / 4, r[2 k + 1] lane t / 4 + 8, column 4 k + t % 4.
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// The upper 16 bits of a float (a bf16, truncated), of two packed, and as a float.
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float top_bits(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

// A piece of one sequence and head (of one role): chunks [c0, c1) in natural order.
struct LaItem {
  const LaRole* r;  // in the kernel's parameters: what a chunk's loop uses is copied out first, since behind
                    // every asm statement it would be loaded again, through memory
  int role, b, h, seg, c0, c1, rev, len;
  int third;  // γ w's third part counts where at most so many tokens follow (-1: nowhere)
  int64_t bh;
  int at;  // chunks of the sequence (or segment) that the walk has behind it
  bool begins, ends;  // the state before it is given (else handed over); the state after it is the end's (else to be handed over)
};

// The k-th piece of this CTA.
__device__ __forceinline__ bool la_item(const LaTcArgs& a, uint32_t k, LaItem& t) {
  const LaParams& p = a.p;
  uint32_t item, p0 = 0, p1 = 0xffffffffu;
  if (!p.balanced) {
    item = blockIdx.x + k * gridDim.x;
    if (item >= a.items) return false;
  } else {
    const uint32_t nch = (uint32_t)p.cps;
    const uint32_t g0 = blockIdx.x * a.share + min(blockIdx.x, a.extra),
                   g1 = g0 + a.share + (blockIdx.x < a.extra ? 1u : 0u);
    const uint32_t first = g0 / nch, r0 = g0 - first * nch, last = g1 / nch, r1 = g1 - last * nch;
    const uint32_t whole0 = first + (r0 != 0), head = r1 != 0;
    if (head && k == 0) {  // the beginning of the sequence that the share ends in
      item = last;
      p1 = r1;
    } else if (k - head < last - whole0) {
      item = whole0 + (k - head);
    } else if (r0 != 0 && k - head == last - whole0) {  // the rest of the one that it begins in
      item = first;
      p0 = r0;
    } else {
      return false;
    }
  }
  const uint32_t rest = item / (uint32_t)p.n_roles, bh = rest / (uint32_t)p.nseg;
  t.role = (int)(item - rest * p.n_roles);
  t.seg = (int)(rest - bh * p.nseg);
  t.bh = bh;
  t.r = &p.role[t.role];
  t.b = (int)(bh / (uint32_t)p.H);
  t.h = (int)bh - t.b * p.H;
  t.rev = t.r->rev;
  // γ^tokens > 2^-6
  t.third = t.r->parts < 3 ? -1 : (int)fminf(__fdividef(6.f, fabsf(p.g[t.h]) * kLog2e), 2e9f);
  t.len = (int)la_len(p, t.b);  // at most 2^30
  la_segment(p, t.len, t.seg, t.rev, t.c0, t.c1);
  t.begins = p0 == 0;
  t.ends = p1 == 0xffffffffu;
  const int n = t.c1 - t.c0, a0 = (int)p0, a1 = t.ends ? n : (int)p1;
  t.at = a0;
  t.c1 = t.c0 + (t.rev ? n - a0 : a1);
  t.c0 = t.c0 + (t.rev ? n - a1 : a0);
  return true;
}

// A state handed from one CTA to the next through global memory: the four warps that write it each add 1 to
// the flag, those that take it wait for 4. The writer has begun with this state, before anything that
// waits, and runs: CTAs start in the order of their indices. The wait is bounded all the same.
__device__ __forceinline__ void hand_over(int* flag, int lane) {
  __threadfence();
  __syncwarp();
  if (lane == 0) atomicAdd(flag, 1);
}
__device__ __forceinline__ bool hand_wait(int* flag, volatile int* abort, int lane) {
  const uint64_t t0 = globaltimer_ns();
  while (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(flag) != 4)) {
    if (__any_sync(0xffffffffu, *abort != 0 || globaltimer_ns() - t0 > kWaitLimitNs)) return false;
  }
  __threadfence();
  return true;
}
// Whether the chunk [t0, t0 + n) needs all three parts.
__device__ __forceinline__ bool la_third(const LaItem& t, int t0, int n) {
  return (t.rev ? t0 : t.len - t0 - n) <= t.third;
}

// First token of the item's chunk number `i` and its count.
__device__ __forceinline__ int la_chunk(const LaItem& t, int i, int& t0) {
  t0 = (t.rev ? t.c1 - 1 - i : t.c0 + i) * kLaChunk;
  return min(kLaChunk, t.len - t0);
}

}  // namespace

// MODE 0: outputs (and the end state, where a sequence is one segment). MODE 1: only every segment's
// end state from zero; needs neither x, nor scores, nor the state's copy.
template <int DX, int DW, int MODE>
__global__ void __launch_bounds__(kThreads, 1) la_tc_kernel(const __grid_constant__ LaTcArgs a) {
  using SM = LaSmem<DX, DW, MODE>;
  constexpr int NX = SM::NX, NY = SM::NY, NW = SM::NW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* x_full = reinterpret_cast<uint64_t*>(sm + SM::BAR);  // [NX] tile landed
  uint64_t* x_empty = x_full + NX;                               // [NX] tile free
  uint64_t* y_full = x_empty + NX;                               // [NY]
  uint64_t* y_empty = y_full + NY;                               // [NY]
  uint64_t* w_full = y_empty + NY;                               // [NW]
  uint64_t* w_empty = w_full + NW;                               // [NW]
  uint64_t* staged = w_empty + NW;                               // [NW] outputs in the W tile
  uint64_t* w_read = staged + NW;                                // [NW] (γ w)ᵀ of the tile has been used
  uint64_t* sc_full = w_read + NW;                             // scores in tensor memory
  uint64_t* p_ready = sc_full + 1;                             // P written, the readout scaled
  uint64_t* m_ready = p_ready + 1;                             // M's copy written
  uint64_t* mx_full = m_ready + 1;                             // the readout in tensor memory; X and the copy free
  uint64_t* o_full = mx_full + 1;                              // P W in tensor memory, P and the tiles free
  uint64_t* o_free = o_full + 1;                               // out columns read
  uint64_t* ring_full = o_free + 1;                            // [RING]
  uint64_t* ring_empty = ring_full + SM::RING;                 // [RING]
  uint64_t* u_full = ring_empty + SM::RING;                    // [NU]
  uint64_t* u_free = u_full + SM::NU;                          // [NU] U read
  uint64_t* pw_full = u_free + SM::NU;                              // [2]
  uint64_t* pw_empty = pw_full + 2;                            // [2]
  // [2] zeros behind a sequence's end written, in turn: warp 1 can be two such chunks ahead of warp 2's wait
  uint64_t* fixed = pw_empty + 2;
  uint64_t* done = fixed + 2;                                  // [2]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + SM::MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + SM::MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LaParams& p = a.p;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NX; ++i) mbar_init(&x_full[i], 1), mbar_init(&x_empty[i], 1);
    for (int i = 0; i < NY; ++i) mbar_init(&y_full[i], 1), mbar_init(&y_empty[i], MODE == 0 ? 2 : 1);
    for (int i = 0; i < NW; ++i) mbar_init(&w_full[i], 1), mbar_init(&w_empty[i], 1), mbar_init(&staged[i], 8), mbar_init(&w_read[i], 1);
    mbar_init(sc_full, 1);
    mbar_init(p_ready, 8);
    mbar_init(m_ready, 4);
    mbar_init(mx_full, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 8);
    for (int i = 0; i < SM::RING; ++i) {
      mbar_init(&ring_full[i], 4 * SM::SUB);
      mbar_init(&ring_empty[i], 1);
    }
    for (int i = 0; i < SM::NU; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_free[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&pw_full[i], 1);
      mbar_init(&pw_empty[i], 16);  // warps 4-11 and 16-23
    }
    mbar_init(&fixed[0], 1);
    mbar_init(&fixed[1], 1);
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The whole warp waits and goes on, or gives up, together.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_wait_warp(bar, parity, abort_flag);
  };
  auto give_up = [&](int where) {
    *abort_flag = 1;
    if (lane == 0) record_device_error(p.status, SWIMBA_ERR_TIMEOUT, where, blockIdx.x, 0);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SM::REG_UTIL));
    if (warp == 0) {
      // ---------------- loads ----------------
      uint32_t it = 0, ii = 0;
      bool ok = true;
      for (LaItem t; ok && la_item(a, ii, t); ++ii) {
        const CUtensorMap* map = a.map[t.role];
        const int hx = t.h / t.r->x.div, hy = t.h / t.r->y.div, hw = t.h / t.r->w.div;
        if (!(ok = wait(&pw_empty[ii & 1], ((ii >> 1) & 1) ^ 1))) break;
        // γ^128, rounded once, would put 1.5e-5 into the state over 512 chunks at a slow decay; in a series of factors
        // it puts 1e-7.
        const float lg = p.g[t.h] * kLog2e;
        const LaDecay g_all = la_decay(p.g[t.h], kLaChunk);
        {
          float* table = reinterpret_cast<float*>(sm + SM::POW) + (ii & 1) * kTable;
          for (int e = lane; e < kTable; e += 32) {
            const int d = t.rev ? kLaChunk - 1 - e : e - 32;
            table[e] = d >= 0 ? la_pow(lg, d) : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&pw_full[ii & 1]);
        }
        for (int i = 0; i < t.c1 - t.c0; ++i, ++it) {
          int t0;
          const int n = la_chunk(t, i, t0);
          const float g = n < kLaChunk ? la_pow(lg, n) : la_factor(g_all, t.at + i);
          auto load = [&](int boxes, int at, const CUtensorMap* m, uint64_t* bar, int head) {
            mbar_arrive_expect_tx(bar, boxes * kTile);
            for (int k = 0; k < boxes; ++k) tma_load_4d(sm + at + k * kTile, m, bar, 64 * k, head, t0, t.b);
          };
          // in the order in which the tiles come free
          if (!(ok = wait(&w_empty[it % NW], ((it / NW) & 1) ^ 1))) break;
          if (elect_one()) {
            *reinterpret_cast<volatile float*>(sm + SM::FACTOR + it % SM::FACTORS * 4) = g;
            load(SM::WB, SM::W + (it % NW) * SM::TW, &map[kMapW], &w_full[it % NW], hw);
          }
          if (!(ok = wait(&y_empty[it % NY], ((it / NY) & 1) ^ 1))) break;
          if (elect_one()) load(SM::XB, SM::Y + (it % NY) * SM::TY, &map[kMapY], &y_full[it % NY], hy);
          if (MODE == 0) {
            if (!(ok = wait(&x_empty[it % NX], ((it / NX) & 1) ^ 1))) break;
            if (elect_one()) load(SM::XB, SM::X + (it % NX) * SM::TX, &map[kMapX], &x_full[it % NX], hx);
          }
          __syncwarp();
        }
      }
      if (!ok) give_up(71);
      // copies that may still be landing (after an orderly end every one has been waited for); `it` counts
      // the chunks whose copies were all issued, the next one's may be
      if (*abort_flag) {
        auto drain = [&](uint64_t* bar, uint32_t n) {
          for (uint32_t k = it + 1 > n ? it + 1 - n : 0; k <= it; ++k) {
            const uint64_t w0 = globaltimer_ns();
            while (!mbar_try_wait(&bar[k % n], (k / n) & 1) && globaltimer_ns() - w0 < kWaitLimitNs / 16) {
            }
          }
        };
        if (MODE == 0) drain(x_full, NX);
        drain(y_full, NY);
        drain(w_full, NW);
      }
    } else if (warp == 2 || (MODE == 0 && warp == 1)) {
      // ---------------- MMAs ----------------
      constexpr uint32_t id_sc = idesc_bf16(128, 128, false), id_mx = idesc_bf16(128, DW, false),
                         id_u = idesc_bf16(128, DX, true), id_pw = idesc_bf16(128, DW, true);
      const uint32_t base = smem_u32(sm);
      // descriptors of address 0, to which a tile's address / 16 is added
      const uint64_t dK = smem_desc(0, 16, 1024, kLayoutSW128), dMN = smem_desc(0, kTile, 1024, kLayoutSW128);
      uint32_t it = 0, ii = 0, fixes = 0;
      bool ok = true;
      for (LaItem t; ok && la_item(a, ii, t); ++ii) {
        for (int i = 0; i < t.c1 - t.c0; ++i, ++it) {
          const uint32_t ph = it & 1;
          int t0;
          const int n = la_chunk(t, i, t0);
          const uint32_t sX = (base + SM::X + (it % NX) * SM::TX) >> 4, sY = (base + SM::Y + (it % NY) * SM::TY) >> 4,
                         sW = (base + SM::W + (it % NW) * SM::TW) >> 4;
          // tokens behind the sequence's end that lie in memory: whatever they hold, they are zeros here
          // (behind the tensor's end the copies have filled in zeros)
          const bool fix = n < kLaChunk && t0 + n < p.L;
          if (!(ok = wait(&y_full[it % NY], (it / NY) & 1))) break;
          if (fix && (MODE == 1 || warp == 1)) {
            if (!(ok = wait(&w_full[it % NW], (it / NW) & 1))) break;
            for (int k = lane; k < (kLaChunk - n) * 8 * (SM::XB + SM::WB); k += 32) {
              const int tile = k / ((kLaChunk - n) * 8), at = k - tile * (kLaChunk - n) * 8;
              uint8_t* s = tile < SM::XB ? sm + SM::Y + (it % NY) * SM::TY + tile * kTile
                                         : sm + SM::W + (it % NW) * SM::TW + (tile - SM::XB) * kTile;
              *reinterpret_cast<uint4*>(s + n * 128 + at * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (MODE == 0 && lane == 0) mbar_arrive(&fixed[fixes & 1]);
            ++fixes;
          }
          if (warp == 2) {
            if (MODE == 0 && fix) {
              if (!(ok = wait(&fixed[fixes & 1], (fixes >> 1) & 1))) break;
              ++fixes;
            }
            // U = Σ_s (γ w_s) y_sᵀ, 16 tokens at a time
            const uint32_t ub = it % SM::NU, up = (it / SM::NU) & 1;
            const bool third = la_third(t, t0, n);
            if (!(ok = wait(&u_free[ub], up ^ 1))) break;
            // A poll queues up behind the MMAs issued before it; asked for after them, it left the tensor cores
            // about 140 cycles without work at every step. So each step's is issued before the MMAs of the
            // step before, and its answer is looked at after them.
            constexpr int R = SM::RING, PER = SM::SLOTS / R;
            bool here = mbar_try_wait(&ring_full[0], (it * PER) & 1);
#pragma unroll 1
            for (int k = 0; k < SM::SLOTS; ++k) {
              if (!__all_sync(0xffffffffu, here) && !(ok = wait(&ring_full[k % R], (it * PER + k / R) & 1))) break;
              tc_fence_after();
              here = k + 1 < SM::SLOTS && mbar_try_wait(&ring_full[(k + 1) % R], (it * PER + (k + 1) / R) & 1);
              if (elect_one()) {
#pragma unroll
                for (int sub = 0; sub < SM::SUB; ++sub)
#pragma unroll
                  for (int part = 0; part < 3; ++part)
                    if (part < 2 || third)
                      mma_bf16_ts(tmem + SM::COL_U + ub * 128,
                                  tmem + SM::COL_RING + ((k % R) * SM::SUB + sub) * 3 * kPart + part * kPart,
                                  dMN + sY + (k * SM::SUB + sub) * (kStep * 8), id_u, (k | sub | part) != 0);
                mma_commit(&ring_empty[k % R]);
                if (k == SM::SLOTS - 1) mma_commit(&u_full[ub]);
              }
              __syncwarp();
            }
            if (!ok) break;
          } else if (MODE == 0) {
            // scores; P of the chunk before has been read
            if (it > 0 && !(ok = wait(o_full, ph ^ 1))) break;
            if (!(ok = wait(&x_full[it % NX], (it / NX) & 1))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll 1
              for (int box = 0; box < SM::XB; ++box)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_bf16(tmem + kColP, dK + sX + box * (kTile >> 4) + k * 2, dK + sY + box * (kTile >> 4) + k * 2, id_sc,
                           (box | k) != 0);
              mma_commit(sc_full);
            }
            __syncwarp();
            // the carried state's readout
            if (!(ok = wait(m_ready, ph))) break;
            if (it > 0 && !(ok = wait(o_free, ph ^ 1))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll 1
              for (int box = 0; box < SM::XB; ++box)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_bf16(tmem + kColO, dK + sX + box * (kTile >> 4) + k * 2,
                           dK + ((base + SM::M) >> 4) + box * (DW * 128 >> 4) + k * 2, id_mx, (box | k) != 0);
              mma_commit(mx_full);
            }
            __syncwarp();
            if (!(ok = wait(&w_full[it % NW], (it / NW) & 1))) break;
            if (!(ok = wait(p_ready, ph))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll 1
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_bf16_ts(tmem + kColO, tmem + kColP + h * 64 + k * 8, dMN + sW + (4 * h + k) * 128, id_pw, 1u);
              mma_commit(o_full);
            }
            __syncwarp();
          }
        }
      }
      if (!ok) give_up(72);
      // every MMA of this warp has completed when its `done` does
      if (elect_one()) {
        mma_commit(&done[warp - 1]);
        const uint64_t w0 = globaltimer_ns();
        while (!mbar_try_wait(&done[warp - 1], 0) && globaltimer_ns() - w0 < kWaitLimitNs) {
        }
      }
      __syncwarp();
    } else if (MODE == 0) {
      // ---------------- stores ----------------
      {
        uint32_t it = 0, ii = 0;
        bool ok = true;
        for (LaItem t; ok && la_item(a, ii, t); ++ii) {
          const bool out_f32 = t.r->out_f32 != 0;
          for (int i = 0; i < t.c1 - t.c0; ++i, ++it) {
            const int st = it % NW;
            int t0;
            const int n = la_chunk(t, i, t0);
            if (!(ok = wait(&staged[st], (it / NW) & 1))) break;
            if (elect_one()) {
              if (!out_f32 && (n == kLaChunk || t0 + n == p.L)) {
#pragma unroll
                for (int k = 0; k < SM::WB; ++k)
                  tma_store_4d(&a.map[t.role][kMapOut], sm + SM::W + st * SM::TW + k * kTile, 64 * k, t.h, t0, t.b);
                bulk_commit();
                bulk_wait_read<0>();
              }
              mbar_arrive(&w_empty[st]);
            }
            __syncwarp();
          }
        }
        if (!ok) give_up(73);
        if (elect_one()) bulk_wait<0>();
        __syncwarp();
      }
    }
  } else if (MODE == 0 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SM::REG_PO));
    {
      // ---------------- scores -> P, outputs ----------------
      const int wq = warp & 3, set = (warp >> 2) - 1, row = 32 * wq + lane;
      const uint32_t tl = tmem + ((uint32_t)(32 * wq) << 16);
      uint32_t it = 0, ii = 0;
      bool ok = true;
      for (LaItem t; ok && la_item(a, ii, t); ++ii) {
        const LaRole& r = *t.r;
        const int rev = t.rev;
        const uint32_t table = smem_u32(sm) + SM::POW + ((ii & 1) * kTable + la_origin(rev) + row) * 4;
        const float s_inter = r.s_inter, s_intra = s_inter * r.s_u, lg = p.g[t.h] * kLog2e;
        const bool out_f32 = r.out_f32 != 0;
        const float f_all = s_inter * la_pow(lg, rev ? kLaChunk - 1 - row : row + 1);
        if (!(ok = wait(&pw_full[ii & 1], (ii >> 1) & 1))) break;
        for (int i = 0; i < t.c1 - t.c0; ++i, ++it) {
          const int st = it % NW;
          const uint32_t ph = it & 1;
          int t0;
          const int n = la_chunk(t, i, t0);
          if (!(ok = wait(sc_full, ph))) break;
          tc_fence_after();
          if (warp == 4 && lane == 0) mbar_arrive(&y_empty[it % NY]);
          // 32 tokens at a time: block blk's bf16 pairs go where this warp's first scores were
#pragma unroll 1
          for (int blk = 2 * set; blk < 2 * set + 2; ++blk) {
            uint32_t w16[16];
            if (rev ? blk >= wq : blk <= wq) {
              float f[32];
              tmem_ld32(tl + kColP + blk * 32, f);
              const uint32_t at = table - blk * 128;
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] *= s_intra * lds1(at - j * 4);
#pragma unroll
              for (int j = 0; j < 16; ++j) w16[j] = pair(f[2 * j], f[2 * j + 1]);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) w16[j] = 0u;
            }
            tmem_st16(tl + kColP + set * 64 + (blk & 1) * 16, w16);
          }
          if (!(ok = wait(mx_full, ph))) break;
          tc_fence_after();
          if (warp == 4 && lane == 0) mbar_arrive(&x_empty[it % NX]);
          const float f_in = rev && n < kLaChunk ? s_inter * la_pow(lg, max(n - 1 - row, 0)) : f_all;
          const uint32_t to = tl + kColO + set * (DW / 2);
#pragma unroll 1
          for (int k = 0; k < DW / 64; ++k) {
            float f[32];
            uint32_t u[32];
            tmem_ld32(to + k * 32, f);
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(f_in * f[j]);
            tmem_st32(to + k * 32, u);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready);
          if (!(ok = wait(&w_read[st], (it / NW) & 1))) break;
          if (!(ok = wait(o_full, ph))) break;
          tc_fence_after();
          const uint32_t tile = smem_u32(sm) + SM::W + st * SM::TW;
          const bool whole = !out_f32 && (n == kLaChunk || t0 + n == p.L);
#pragma unroll 1
          for (int k = 0; k < DW / 64; ++k) {
            float f[32];
            tmem_ld32(to + k * 32, f);
            const int b32 = set * (DW / 64) + k;  // 32 columns of the tile
            if (whole) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                sts4(tile + (b32 >> 1) * kTile + swz16(row, (b32 & 1) * 4 + c), pair(f[8 * c], f[8 * c + 1]),
                     pair(f[8 * c + 2], f[8 * c + 3]), pair(f[8 * c + 4], f[8 * c + 5]), pair(f[8 * c + 6], f[8 * c + 7]));
            } else if (row < n) {
              const int dw = r.dw;
              void* const out = r.out;
              const int64_t at = t.b * r.out_sb + (t0 + row) * r.out_st + (int64_t)t.h * dw;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int col = b32 * 32 + 8 * c;
                if (col >= dw) continue;
                if (out_f32) {
                  float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at + col);
                  dst[0] = make_float4(f[8 * c], f[8 * c + 1], f[8 * c + 2], f[8 * c + 3]);
                  dst[1] = make_float4(f[8 * c + 4], f[8 * c + 5], f[8 * c + 6], f[8 * c + 7]);
                } else {
                  *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + at + col) =
                      make_uint4(pair(f[8 * c], f[8 * c + 1]), pair(f[8 * c + 2], f[8 * c + 3]),
                                 pair(f[8 * c + 4], f[8 * c + 5]), pair(f[8 * c + 6], f[8 * c + 7]));
                }
              }
            }
            __syncwarp();
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(o_free);
            mbar_arrive(&staged[st]);
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&pw_empty[ii & 1]);
      }
      if (!ok) give_up(75);
    }
  } else if (warp >= 12 && warp < 16) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SM::REG_M));
    // ---------------- the state ----------------
    const int wq = warp & 3, col = 32 * wq + lane;  // column of M = lane of U
    const uint32_t tl = tmem + ((uint32_t)(32 * wq) << 16);
    const bool active = col < DW;  // the same for a whole warp
    uint32_t it = 0, ii = 0;
    bool ok = true;
    for (LaItem t; ok && la_item(a, ii, t); ++ii) {
      const LaRole& r = *t.r;
      const int dx = r.dx, dw = r.dw;
      const int64_t size = (int64_t)dx * dw;
      float m[DX];
      {
        const float* start = MODE == 1     ? nullptr
                             : !t.begins   ? p.hand_states + (size_t)(blockIdx.x - 1) * 128 * 128
                             : p.nseg > 1  ? r.seg + (t.bh * p.nseg + t.seg) * size
                             : r.M0        ? r.M0 + t.bh * size
                                           : nullptr;
        const bool own = t.begins && p.nseg == 1;  // in the caller's layout, else [dx, dw]
        if (!t.begins && !(ok = hand_wait(&p.hand_flags[blockIdx.x - 1], abort_flag, lane))) break;
        if (start != nullptr && col < dw) {
          const int sj = own ? r.sj : dw;
          const float* from = start + (int64_t)col * (own ? r.sc : 1);
#pragma unroll
          for (int j = 0; j < DX; ++j, from += sj) m[j] = j < dx ? __ldcg(from) : 0.f;
        } else {
#pragma unroll
          for (int j = 0; j < DX; ++j) m[j] = 0.f;
        }
      }
      // M's bf16 copy; the readout of the chunk before has taken the last one
      auto copy = [&]() {
        if (active) {
#pragma unroll
          for (int c = 0; c < DX / 8; ++c)
            sts4(smem_u32(sm) + SM::M + (c >> 3) * (DW * 128) + swz16(col, c & 7), pair(m[8 * c], m[8 * c + 1]),
                 pair(m[8 * c + 2], m[8 * c + 3]), pair(m[8 * c + 4], m[8 * c + 5]), pair(m[8 * c + 6], m[8 * c + 7]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(m_ready);
      };
      const int chunks = t.c1 - t.c0;
#pragma unroll 1
      for (int i = 0; i < chunks; ++i, ++it) {
        if (MODE == 0) {
          if (it > 0 && !(ok = wait(mx_full, (it & 1) ^ 1))) break;
          copy();
        }
        const uint32_t ub = it % SM::NU;
        if (!(ok = wait(&u_full[ub], (it / SM::NU) & 1))) break;
        tc_fence_after();
        // written before W's copy was issued, which U has waited for
        const float g = lds1(smem_u32(sm) + SM::FACTOR + it % SM::FACTORS * 4);
        if (wq == 0 && lane == 0) {
          mbar_arrive(&y_empty[it % NY]);
          mbar_arrive(MODE == 0 ? &w_read[it % NW] : &w_empty[it % NW]);
        }
        if (active) {
#pragma unroll
          for (int k = 0; k < DX / 16; ++k) {
            float f[16];
            tmem_ld16(tl + SM::COL_U + ub * 128 + k * 16, f);
#pragma unroll
            for (int j = 0; j < 16; ++j) m[k * 16 + j] = fmaf(g, m[k * 16 + j], f[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_free[ub]);
      }
      if (!ok) break;
      const bool hand = MODE == 0 && !t.ends;
      float* end = MODE == 1                              ? r.seg + (t.bh * p.nseg + t.seg) * size
                   : hand                                 ? p.hand_states + (size_t)blockIdx.x * 128 * 128
                   : p.nseg == 1 && r.M_end != nullptr    ? r.M_end + t.bh * size
                                                          : nullptr;
      if (end != nullptr && col < dw) {
        const bool own = MODE == 0 && !hand;
        const int ej = own ? r.sj : dw;
        end += (int64_t)col * (own ? r.sc : 1);
#pragma unroll
        for (int j = 0; j < DX; ++j, end += ej)
          if (j < dx) *end = m[j];
      }
      if (hand) hand_over(&p.hand_flags[blockIdx.x], lane);
    }
    if (!ok) give_up(76);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SM::REG_W));
    // ---------------- (γ w)ᵀ ----------------
    const int wq = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(32 * wq) << 16);
    const bool active = 32 * wq < DW;
    const int set = warp >= 16 ? (warp >> 2) - 4 : (warp >> 2) + 1;  // 16-19, 20-23, then 4-7, 8-11
    if (!active) {  // those rows stay zero
      const uint32_t z[8] = {};
#pragma unroll 1
      for (int k = 0; k < SM::RING * SM::SUB * 3; ++k) tmem_st8(tl + SM::COL_RING + k * kPart, z);
      tmem_wait_st();
    }
    uint32_t it = 0, ii = 0;
    bool ok = true;
    for (LaItem t; ok && la_item(a, ii, t); ++ii) {
      const int rev = t.rev;
      const uint32_t table = smem_u32(sm) + SM::POW + ((ii & 1) * kTable + la_origin(rev)) * 4;
      const float f_w = rev ? t.r->s_u * la_pow(p.g[t.h] * kLog2e, 1) : t.r->s_u;
      if (!(ok = wait(&pw_full[ii & 1], (ii >> 1) & 1))) break;
      for (int i = 0; i < t.c1 - t.c0; ++i, ++it) {
        const int st = it % NW;
        int t0;
        const int n = la_chunk(t, i, t0);
        const bool third = la_third(t, t0, n);
        if (!(ok = wait(&w_full[st], (it / NW) & 1))) break;
        // 16 tokens at a time: 8 x 8 blocks of W, transposed on the way to the registers, where thread t
        // holds channel t / 4 of tokens 2 (t % 4) + 0..1, scaled, split and stored in that form
        const uint32_t tw = smem_u32(sm) + SM::W + st * SM::TW + (wq >> 1) * kTile + ((lane & 7) + 8 * (lane >> 4)) * 128;
#pragma unroll 1
        for (int k = set / SM::SUB; k < SM::SLOTS; k += SM::GROUPS) {
          constexpr int R = SM::RING, PER = SM::SLOTS / R;
          const uint32_t slot = k % R;
          if (!(ok = wait(&ring_empty[slot], ((it * PER + k / R) & 1) ^ 1))) break;
          tc_fence_after();
          if (active) {
            const int sub = set % SM::SUB, step = k * SM::SUB + sub;
            uint32_t raw[2][4];
#pragma unroll
            for (int half = 0; half < 2; ++half)  // 16 channels: matrices (tokens, channels) (0, 0), (0, 8), (8, 0), (8, 8)
              ldmatrix_x4_trans(tw + step * (kStep * 128) + ((((wq & 1) * 4 + half * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4),
                                raw[half]);
            float2 wt[2];
            uint32_t keep[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              // γ^(n-1-s), reverse γ γ^s; tokens behind the last chunk's end count as zeros whatever they hold
              const int s = kStep * step + 8 * g + 2 * (lane & 3), e = rev ? s : max(n - 2 - s, -1);
              const float a0 = lds1(table + (rev ? -e : e + 1) * 4), a1 = lds1(table + (rev ? -e - 1 : e) * 4);
              wt[g] = make_float2(a0 * f_w, a1 * f_w);
              keep[g] = (s < n ? 0xffffu : 0u) | (s + 1 < n ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t hi[4], mid[4], lo[4];
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                // three truncated parts of 8 bits each: their sum is the product's 24 bits
                const uint32_t v = raw[half][d] & keep[d >> 1];
                const float v0 = bf16lo(v) * wt[d >> 1].x, v1 = bf16hi(v) * wt[d >> 1].y;
                hi[d] = high_halves(v0, v1);
                const float r0 = v0 - top_bits(v0), r1 = v1 - top_bits(v1);
                mid[d] = high_halves(r0, r1);
                lo[d] = high_halves(r0 - top_bits(r0), r1 - top_bits(r1));
              }
              const uint32_t at = tl + ((uint32_t)(16 * half) << 16) + SM::COL_RING + (slot * SM::SUB + sub) * 3 * kPart;
              tmem_st_16x128b_x2(at, hi);
              tmem_st_16x128b_x2(at + kPart, mid);
              if (third) tmem_st_16x128b_x2(at + 2 * kPart, lo);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ring_full[slot]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&pw_empty[ii & 1]);
    }
    if (!ok) give_up(77);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- host -----------------------------------------------------------------------------------------------
namespace {

PFN_cuTensorMapEncodeTiled_v12000 la_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// [B, L, heads, d] bf16 with token stride st: boxes of 128 tokens x 64 channels of one head; what lies
// behind d or L reads as zeros and is not written.
bool la_map(CUtensorMap* m, const void* base, int d, int heads, int64_t st, int64_t L, int64_t B) {
  auto fn = la_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)B};
  cuuint64_t str[3] = {(cuuint64_t)(d * 2), (cuuint64_t)(st * 2), (cuuint64_t)(st * L * 2)};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)kLaChunk, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, str, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DX, int DW, int MODE>
cudaError_t launch_tc(const LaTcArgs& a, int sms, cudaStream_t s) {
  constexpr int smem = 1024 + LaSmem<DX, DW, MODE>::BYTES;
  const cudaError_t e = cudaFuncSetAttribute(la_tc_kernel<DX, DW, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  la_tc_kernel<DX, DW, MODE><<<(unsigned)std::min<uint32_t>(a.items, sms), kThreads, smem, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

// One launch over roles of the same padded sizes. states: only the segments' end states.
cudaError_t run_la_tc(const LaParams& p, bool states, cudaStream_t s) {
  LaTcArgs a;
  a.p = p;
  a.items = (uint32_t)p.n_roles * p.B * p.H * p.nseg;  // below 2^30
  for (int i = 0; i < p.n_roles; ++i) {
    const LaRole& r = p.role[i];
    if (!la_map(&a.map[i][kMapX], r.x.p, r.dx, p.H / r.x.div, r.x.st, p.L, p.B) ||
        !la_map(&a.map[i][kMapY], r.y.p, r.dx, p.H / r.y.div, r.y.st, p.L, p.B) ||
        !la_map(&a.map[i][kMapW], r.w.p, r.dw, p.H / r.w.div, r.w.st, p.L, p.B) ||
        (!r.out_f32 && !la_map(&a.map[i][kMapOut], r.out, r.dw, p.H, r.out_st, p.L, p.B)))
      return cudaErrorInvalidValue;
  }
  int dev = 0, sms = kLaCtas;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  sms = std::min(sms, kLaCtas);
  // Equal shares cut sequences; they pay where whole ones would leave CTAs idle in the last round, and
  // need at least as many pieces as CTAs, so that a sequence spans two shares at most. With lengths on
  // the device the host does not know the shares.
  const uint64_t total = (uint64_t)a.items * p.cps, rounds = (a.items + sms - 1) / sms;
  a.share = (uint32_t)(total / sms);
  a.extra = (uint32_t)(total % sms);
  a.p.balanced = !states && p.hand_flags != nullptr && p.nseg == 1 && p.lens == nullptr && a.items >= (uint32_t)sms &&
                 total < (1u << 31) && (double)(rounds * p.cps) > la_shared_units((int64_t)total, sms);
  if (a.p.balanced) {
    const cudaError_t e = cudaMemsetAsync(p.hand_flags, 0, kLaFlagBytes, s);
    if (e != cudaSuccess) return e;
  }
  const bool x64 = p.role[0].dx <= 64, w64 = p.role[0].dw <= 64;
  if (states)
    return x64 ? (w64 ? launch_tc<64, 64, 1>(a, sms, s) : launch_tc<64, 128, 1>(a, sms, s))
               : (w64 ? launch_tc<128, 64, 1>(a, sms, s) : launch_tc<128, 128, 1>(a, sms, s));
  return x64 ? (w64 ? launch_tc<64, 64, 0>(a, sms, s) : launch_tc<64, 128, 0>(a, sms, s))
             : (w64 ? launch_tc<128, 64, 0>(a, sms, s) : launch_tc<128, 128, 0>(a, sms, s));
}

}  // namespace swimba
