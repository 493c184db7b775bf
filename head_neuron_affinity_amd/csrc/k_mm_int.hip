// 8-bit integer product on the matrix cores:
//   out[t, n] = (sum_k q[t, k] w[n, k]) q_scale[t] w_scale[n]
// q [T, K] and w [N, K] row-major with k contiguous, sums in int32 (exact for
// K < 2^17), the scales applied in fp32, one rounding to the output type.
// The channels are the MFMA rows and the tokens its columns, so a lane ends up
// with 4 consecutive channels of one token: out's contiguous direction.
// Tiles of 128 x 128 on 4 waves, 128 bytes of k a step through LDS.
#include "hna_internal.h"
#include "hna_hot.h"

namespace hna {
namespace {

using namespace hot;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

__device__ inline void mma_int(i32x16& c, const uint4& a, const uint4& b) {
  c = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// 4 consecutive channels n .. n + 3 of token t
__device__ inline void put4(const IntMmParams& p, int64_t t, int n, const int (&v)[4], float st) {
  const int64_t o = t * p.N + n;
  if (n + 4 <= p.N && p.N % 4 == 0) {
    const float4 sw = *reinterpret_cast<const float4*>(p.w_scale + n);
    const float f[4] = {(float)v[0] * st * sw.x, (float)v[1] * st * sw.y, (float)v[2] * st * sw.z, (float)v[3] * st * sw.w};
    if (p.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(f[0], f[1], f[2], f[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    const float f = (float)v[e] * st * p.w_scale[n + e];
    if (p.out_bf16) static_cast<uint16_t*>(p.out)[o + e] = (uint16_t)pack_bf16x2(f, 0.f);
    else static_cast<float*>(p.out)[o + e] = f;
  }
}

template <int BM, int BN, int WGM, int WGN, int NST>
__global__ __launch_bounds__(64 * WGM * WGN) void mm_int_kernel(const IntMmParams p) {
  constexpr int NW = WGM * WGN;
  constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  constexpr int ROWS = BM + BN, BK = 128, CPR = BK / 16, RPI = 64 / CPR;
  constexpr int STAGE = ROWS * BK;
  constexpr int NCP = ROWS / (RPI * NW), NCX = BM / (RPI * NW);
  static_assert(BM % (RPI * NW) == 0 && BN % (RPI * NW) == 0, "copy rounds cover whole rows");
  static_assert((NST - 2) * NCP <= 63, "copies in flight must fit the wait counter");
  __shared__ __attribute__((aligned(16))) unsigned char lds[NST * STAGE];

  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WGN, wn = w % WGN;

  // tile of this workgroup: XCD by XCD, in groups of 4 tile rows
  const int ntm = (p.N + BM - 1) / BM;
  const int64_t ntn = (p.T + BN - 1) / BN, ntiles = ntm * ntn;
  const int64_t per_xcd = (ntiles + 7) / 8;
  const int64_t t = (int64_t)(blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per_xcd || t >= ntiles) return;
  constexpr int GM = 4;
  const int64_t gsize = GM * ntn;
  const int g0 = (int)(t / gsize) * GM, gm = min(GM, ntm - g0);
  const int64_t tg = t - (t / gsize) * gsize;
  const int n0 = (g0 + (int)(tg % gm)) * BM;
  const int64_t t0 = tg / gm * BN;

  const int64_t xb = (int64_t)(p.N - n0) * p.K, yb = (p.T - t0) * p.K;
  const u32x4 rx = uniform_rsrc(p.w + (int64_t)n0 * p.K, xb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)xb);
  const u32x4 ry = uniform_rsrc(p.q + t0 * p.K, yb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)yb);

  i32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x16{};
  const int nk = (p.K + BK - 1) / BK;

  // copy i of wave w fills rows RPI (NW i + w) .. + RPI - 1 of the stage (w
  // rows first); rows past the end and bytes past K read zeros
  uint32_t voff[NCP];
  int kc[NCP];
#pragma unroll
  for (int i = 0; i < NCP; ++i) {
    const int r = RPI * (NW * i + w) + l / CPR;
    kc[i] = 16 * ((l % CPR) ^ swz<CPR>(r));
    voff[i] = (uint32_t)((int64_t)(i < NCX ? r : r - BM) * p.K + kc[i]);
  }
  const uint32_t lds0 = lds_addr(lds) + (uint32_t)w * 1024u;
  auto issue = [&](int k0, int buf) __attribute__((always_inline)) {
    const uint32_t base = lds0 + (uint32_t)(buf * STAGE);
    const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)k0);
#pragma unroll
    for (int i = 0; i < NCP; ++i)
      dma16s(i < NCX ? rx : ry, k0 + kc[i] >= p.K ? kOutOfRange : voff[i], soff, base + (uint32_t)(i * NW * 1024));
  };

#pragma unroll
  for (int st = 0; st < NST - 1; ++st)
    if (st < nk) issue(st * BK, st);
  for (int kt = 0; kt < nk; ++kt) {
    // step kt has landed once at most the copies of the steps after it are in
    // flight; the barrier shows it to every wave and ends their reads of step kt - 1
    const int ahead = min(NST - 2, nk - 1 - kt);
    if (NST >= 4 && ahead >= 2) __builtin_amdgcn_s_waitcnt(vm_wait(2 * NCP));
    else if (NST >= 3 && ahead >= 1) __builtin_amdgcn_s_waitcnt(vm_wait(NCP));
    else __builtin_amdgcn_s_waitcnt(vm_wait(0));
    __syncthreads();
    if (kt + NST - 1 < nk) issue((kt + NST - 1) * BK, (kt + NST - 1) % NST);
    const unsigned char* sb = lds + (kt % NST) * STAGE;
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks) {
      const int col = 2 * ks + (l >> 5);
      uint4 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = wm * WM + i * 32 + (l & 31);
        fa[i] = *reinterpret_cast<const uint4*>(sb + r * BK + ((col ^ swz<CPR>(r)) << 4));
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int r = BM + wn * WN + j * 32 + (l & 31);
        fb[j] = *reinterpret_cast<const uint4*>(sb + r * BK + ((col ^ swz<CPR>(r)) << 4));
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) mma_int(acc[i][j], fa[i], fb[j]);
    }
  }

  // lane l holds token (l & 31) and channels 8 (v / 4) + 4 (l / 32) + v % 4 of each tile
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t tk = t0 + wn * WN + j * 32 + (l & 31);
    if (tk >= p.T) continue;
    const float st = p.q_scale[tk];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int n = n0 + wm * WM + i * 32 + 8 * a + 4 * (l >> 5);
        if (n >= p.N) continue;
        const int v[4] = {acc[i][j][4 * a], acc[i][j][4 * a + 1], acc[i][j][4 * a + 2], acc[i][j][4 * a + 3]};
        put4(p, tk, n, v, st);
      }
  }
}

// Large products: a 256 x 256 tile on 4 waves, one per SIMD, each 128 x 128
// (16 accumulators of 32 x 32: the largest wave tile, so that the fragment
// reads and the copies together keep LDS busy 3/4 of the MFMA time).  64 bytes
// of k a step in a ring of four stages.  A step is two halves of 32 bytes; the
// fragments of the next half are read while the MFMAs of this one run:
//   MFMA half 0, reading half 1 of step k
//   wait for the reads and for step k + 1's copies; barrier
//   MFMA half 1, reading half 0 of step k + 1, copying step k + 4 over step k
// The barrier says that every wave holds step k in registers (its buffer is
// free) and that every wave's part of step k + 1 is in LDS.  Copies past K read
// zeros, so the loop needs no tail.
__global__ __launch_bounds__(256, 1) void mm_int_big_kernel(const IntMmParams p) {
  constexpr int BM = 256, BN = 256, BK = 128, NST = 2, STAGE = (BM + BN) * BK;
  __shared__ __attribute__((aligned(16))) unsigned char lds[NST * STAGE];
  __shared__ __attribute__((aligned(16))) float sw[BM];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w >> 1, wn = w & 1;

  const int ntm = (p.N + BM - 1) / BM;
  const int64_t ntn = (p.T + BN - 1) / BN, ntiles = ntm * ntn;
  const int64_t per_xcd = (ntiles + 7) / 8;
  const int64_t t = (int64_t)(blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per_xcd || t >= ntiles) return;
  constexpr int GM = 4;
  const int64_t gsize = GM * ntn;
  const int g0 = (int)(t / gsize) * GM, gm = min(GM, ntm - g0);
  const int64_t tg = t - (t / gsize) * gsize;
  const int n0 = (g0 + (int)(tg % gm)) * BM;
  const int64_t t0 = tg / gm * BN;

  const int64_t xb = (int64_t)(p.N - n0) * p.K, yb = (p.T - t0) * p.K;
  const u32x4 rx = uniform_rsrc(p.w + (int64_t)n0 * p.K, xb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)xb);
  const u32x4 ry = uniform_rsrc(p.q + t0 * p.K, yb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)yb);

  // a stage holds rows of 128 bytes (whole cache lines: copies of 64 bytes a row
  // took twice the L2 requests and 1.2 times as long), chunk c of row r in slot
  // c ^ swz(r).  Copy i of wave w fills rows 32 i + 8 w + l / 8.
  const int kc = 16 * ((l & 7) ^ swz<8>(8 * w + (l >> 3)));
  uint32_t voff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) voff[i] = (uint32_t)((32 * i + 8 * w + (l >> 3)) * p.K + kc);
  const uint32_t lds0 = lds_addr(lds) + (uint32_t)w * 1024u;
  // copy c of 16 of step kt: rows 32 (c / 2) + .. of w (c even) or q (c odd)
  auto issue = [&](int kt, int c) __attribute__((always_inline)) {
    const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)(kt * BK));
    const uint32_t v = kt * BK + kc >= p.K ? kOutOfRange : voff[c >> 1];
    dma16s(c & 1 ? ry : rx, v, soff,
           lds0 + (uint32_t)((kt & (NST - 1)) * STAGE + (c & 1) * BM * BK + (c >> 1) * 4096));
  };
  i32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = i32x16{};
  uint4 fa[2][4], fb[2][4];
  const int sl = swz<8>(l & 31), up = l >> 5;
  const int ra = (wm * 128 + (l & 31)) * BK, rb = (BM + wn * 128 + (l & 31)) * BK;
  // fragment f of 8 (4 of the channels, 4 of the tokens) of quarter h of step kt
  auto rd = [&](int kt, auto h, int f) __attribute__((always_inline)) {
    const unsigned char* sb = lds + (kt & (NST - 1)) * STAGE + (((2 * h + up) ^ sl) << 4);
    if (f < 4) fa[h & 1][f] = *reinterpret_cast<const uint4*>(sb + ra + f * 32 * BK);
    else fb[h & 1][f - 4] = *reinterpret_cast<const uint4*>(sb + rb + (f - 4) * 32 * BK);
  };
  // the 16 MFMAs of quarter h, after(i) right behind the i-th
  auto mm = [&](auto quarter, auto after) __attribute__((always_inline)) {
    constexpr int h = decltype(quarter)::value & 1;
    static_for<0, 16>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      mma_int(acc[i / 4][i % 4], fa[h][i / 4], fb[h][i % 4]);
      after(ic);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  constexpr std::integral_constant<int, 0> Q0{};
  constexpr std::integral_constant<int, 1> Q1{};
  constexpr std::integral_constant<int, 2> Q2{};
  constexpr std::integral_constant<int, 3> Q3{};

  sw[tid] = n0 + tid < p.N ? p.w_scale[n0 + tid] : 0.f;   // read after the loop's barriers
  const int nk = (p.K + BK - 1) / BK;
#pragma unroll
  for (int s = 0; s < NST; ++s)
#pragma unroll
    for (int c = 0; c < 16; ++c) issue(s, c);
  __builtin_amdgcn_s_waitcnt(vm_wait(16));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int f = 0; f < 8; ++f) rd(0, Q0, f);
  for (int kt = 0; kt < nk; ++kt) {
    mm(Q0, [&](auto i) __attribute__((always_inline)) {
      if constexpr (i < 8) rd(kt, Q1, i);
    });
    mm(Q1, [&](auto i) __attribute__((always_inline)) {
      if constexpr (i < 8) rd(kt, Q2, i);
    });
    mm(Q2, [&](auto i) __attribute__((always_inline)) {
      if constexpr (i < 8) rd(kt, Q3, i);
    });
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    mm(Q3, [&](auto i) __attribute__((always_inline)) {
      if constexpr (i < 8) rd(kt + 1, Q0, i);
      issue(kt + NST, i);
    });
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);

  // lane l holds token (l & 31) and channels 8 a + 4 (l / 32) + e of each tile:
  // scaled, rounded and staged through this wave's quarter of LDS, 32 tokens x
  // 128 channels at a time, so that out is written in full runs of a token's
  // 128 channels
  unsigned char* stg = lds + w * (NST * STAGE / 4);
  const int nw = n0 + wm * 128;
  auto write = [&](auto bf16) __attribute__((always_inline)) {
    constexpr int E = decltype(bf16)::value ? 2 : 4;      // bytes per output
    constexpr int PITCH = 128 * E + 16;
    static_assert(32 * PITCH <= NST * STAGE / 4, "staging fits");
    constexpr int PER = 16 / E, LPR = 128 / PER, RPW = 64 / LPR;   // outputs and lanes per 16 bytes, rows per store
    const bool wide = p.N % PER == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t tj = t0 + wn * 128 + j * 32;
      const float st = tj + (l & 31) < p.T ? p.q_scale[tj + (l & 31)] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int n = i * 32 + 8 * a + 4 * up;
          const float4 s4 = *reinterpret_cast<const float4*>(sw + wm * 128 + n);
          const float f[4] = {(float)acc[i][j][4 * a] * st * s4.x, (float)acc[i][j][4 * a + 1] * st * s4.y,
                              (float)acc[i][j][4 * a + 2] * st * s4.z, (float)acc[i][j][4 * a + 3] * st * s4.w};
          unsigned char* d = stg + (l & 31) * PITCH + n * E;
          if constexpr (E == 2) *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
          else *reinterpret_cast<float4*>(d) = make_float4(f[0], f[1], f[2], f[3]);
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int k = 0; k < 32 / RPW; ++k) {
        const int row = k * RPW + l / LPR, c = (l % LPR) * PER;
        if (tj + row >= p.T || nw + c >= p.N) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(stg + row * PITCH + c * E);
        unsigned char* o = static_cast<unsigned char*>(p.out) + ((tj + row) * p.N + nw + c) * E;
        if (wide) {
          *reinterpret_cast<uint4*>(o) = v;
        } else {
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
          const int m = min(PER, p.N - nw - c);
          for (int e = 0; e < m; ++e) {
            if constexpr (E == 2) reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
            else reinterpret_cast<uint32_t*>(o)[e] = u[e];
          }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  };
  if (p.out_bf16) write(std::true_type{});
  else write(std::false_type{});
}

template <int BM, int BN, int WGM, int WGN, int NST>
hipError_t launch_t(const IntMmParams& p, hipStream_t st) {
  const int64_t ntiles = (int64_t)((p.N + BM - 1) / BM) * ((p.T + BN - 1) / BN);
  const dim3 grid((unsigned)(8 * ((ntiles + 7) / 8)));
  hipLaunchKernelGGL((mm_int_kernel<BM, BN, WGM, WGN, NST>), grid, dim3(64 * WGM * WGN), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_int(const IntMmParams& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  const int64_t tiles = (int64_t)((p.N + 255) / 256) * ((p.T + 255) / 256);
  if (tiles >= 256) {
    hipLaunchKernelGGL(mm_int_big_kernel, dim3((unsigned)(8 * ((tiles + 7) / 8))), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  return launch_t<128, 128, 2, 2, 2>(p, st);
}

}  // namespace hna
