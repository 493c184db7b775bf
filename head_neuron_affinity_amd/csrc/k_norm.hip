// The norm step between two blocks, and its gradients.
//
//   b  = y / r_post * gamma_post (r_post = sqrt(mean y^2 + eps)), or y;  b *= gate
//   x' = res_scale x + block_scale b, rounded to the residual's type
//   n  = gamma x' / r,  r = sqrt(mean x'^2 + eps),  of x' as stored;
//        or n as 8-bit integers with one scale per token
//
// One pass over the data: NT lanes hold a row in registers (CH chunks of 8
// elements each), so x' and y are read once and n needs no second read.  Sums
// run in fp32 over 8 CH elements per lane, then across lanes in a fixed order.
// Bound by HBM (65536 x 4096 bf16 0.364 to 0.397 ms, 5.4 to 5.9 TB/s; the next row loaded
// ahead made it 0.435).  A row sits in one wave up to 1024 elements (no
// barrier), in NT / 64 waves above; a workgroup walks over rows with the gains
// in registers.
#include <algorithm>

#include "hna_rows.h"

namespace hna {
namespace {

using namespace rows;

constexpr int wg_of(int nt) { return nt < 256 ? 256 : nt; }

// 1 / r, or 0 for a row whose mean square and eps are both 0: it normalises to zeros
__device__ inline float inv_or_zero(float r) { return r > 0.f ? 1.f / r : (r == 0.f ? 0.f : r); }

// S: past the caches (see streams)
template <typename R, typename D, int NT, int CH, bool Q8, bool S>
__global__ __launch_bounds__(wg_of(NT)) void block_norm_kernel(const NormParams p) {
  constexpr int WG = wg_of(NT), NR = WG / NT;
  constexpr bool SPLIT = sizeof(R) == 4 || sizeof(D) == 4;
  __shared__ uint32_t box[2 * (WG / 64)];
  int phase = 0;
  const Lane<NT, SPLIT> ln{(int)threadIdx.x % NT};
  const int sub = threadIdx.x / NT, C = p.C;
  const float inv_c = 1.f / (float)C;

  float ga[CH][8], gp[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_gain(p.gamma, ln, c, p.gamma ? C : 0, ga[c]);
    load_gain(p.gamma_post, ln, c, p.gamma_post ? C : 0, gp[c]);
  }

  for (int64_t row0 = (int64_t)blockIdx.x * NR; row0 < p.T; row0 += (int64_t)gridDim.x * NR) {
    const int64_t row = row0 + sub;
    const bool live = row < p.T;
    const int64_t base = row * C;
    float h[CH][8], y[CH][8];
    {
      Raw8<R, SPLIT> rx[CH];
      Raw8<D, SPLIT> ry[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        rx[c].template load<S>(static_cast<const R*>(p.x) + base, ln, c, C, live);
        ry[c].template load<S>(static_cast<const D*>(p.y) + base, ln, c, C, live && p.y);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        rx[c].get(h[c]);
        ry[c].get(y[c]);
      }
    }
    if (p.y) {
      float m = p.block_scale;
      if (p.gamma_post) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(y[c][e], y[c][e], s);
        const float rp = sqrtf(fmaf(row_sum<NT, WG>(s, box, phase), inv_c, p.eps));
        if (live && ln.lane == 0 && p.r_post) p.r_post[row] = rp;
        m *= inv_or_zero(rp);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = gp[c][e];
        if (p.gate) {
          float v[8];
          Raw8<D, SPLIT> rg;
          rg.template load<false>(static_cast<const D*>(p.gate) + (live ? (int64_t)((uint32_t)row / (uint32_t)p.gate_tokens) * C : 0),
                                  ln, c, C, live);
          rg.get(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= v[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          h[c][e] = as_stored<R>(fmaf(p.res_scale, h[c][e], y[c][e] * m * g[e]));
        if (live) store8<S>(static_cast<R*>(p.x_out) + base, ln, c, C, h[c]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(h[c][e], h[c][e], s);
    const float r = sqrtf(fmaf(row_sum<NT, WG>(s, box, phase), inv_c, p.eps));
    if (live && ln.lane == 0 && p.r) p.r[row] = r;
    const float inv = inv_or_zero(r);
    if constexpr (!Q8) {
      if (!p.n) continue;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = h[c][e] * inv * ga[c][e];
        if (live) store8<S>(static_cast<D*>(p.n) + base, ln, c, C, v);
      }
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[c][e] = ln.at(c, e >> 2) < C ? h[c][e] * inv * ga[c][e] : 0.f;
          top = max_bits(top, __float_as_uint(h[c][e]) & 0x7fffffffu);
        }
      const RowScale rs = row_scale(row_max_bits<NT, WG>(top, box, phase));
      if (live && ln.lane == 0) p.q_scale[row] = rs.scale;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (live) store_quant8(p.q + row * p.pitch, ln, c, p.pitch, quant8(h[c], rs));
    }
  }
}

// Rows of x as 8-bit integers.  VEC: rows start on 16 bytes.  Bound by HBM: 65536
// x 1536 bf16 51 us, 5.9 TB/s; 16384 x 14336 113 us, 6.2 TB/s.  Otherwise by loads
// of one element a lane: 16384 x 14331 bf16 456 us, 1.5 TB/s, 4096 x 14331 fp32 63
// us, 4.7 TB/s.
template <typename D, int NT, int CH, bool VEC, bool S>
__global__ __launch_bounds__(wg_of(NT)) void quant_rows_kernel(const D* __restrict__ x, int64_t n_rows,
                                                               int K, int pitch, int8_t* __restrict__ q,
                                                               float* __restrict__ scale) {
  constexpr int WG = wg_of(NT), NR = WG / NT;
  constexpr bool SPLIT = sizeof(D) == 4;
  __shared__ uint32_t box[2 * (WG / 64)];
  int phase = 0;
  const Lane<NT, SPLIT> ln{(int)threadIdx.x % NT};
  const int sub = threadIdx.x / NT;
  for (int64_t row0 = (int64_t)blockIdx.x * NR; row0 < n_rows; row0 += (int64_t)gridDim.x * NR) {
    const int64_t row = row0 + sub;
    const bool live = row < n_rows;
    const D* xr = x + row * K;
    float v[CH][8];
    if constexpr (VEC) {
      Raw8<D, SPLIT> raw[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) raw[c].template load<S>(xr, ln, c, K, live);
#pragma unroll
      for (int c = 0; c < CH; ++c) raw[c].get(v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = ln.at(c, e >> 2) + (e & 3);
          v[c][e] = live && j < K ? (float)xr[j] : 0.f;
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_bits(top, __float_as_uint(v[c][e]) & 0x7fffffffu);
    const RowScale rs = row_scale(row_max_bits<NT, WG>(top, box, phase));
    if (live && ln.lane == 0) scale[row] = rs.scale;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (live) store_quant8(q + row * pitch, ln, c, pitch, quant8(v[c], rs));
  }
}

// Rows too long for registers (K > 16384): read twice, one workgroup per row, an
// element a lane: 8192 x 28672 bf16 463 us, 1.5 TB/s.
template <typename D>
__global__ __launch_bounds__(1024) void quant_long_rows_kernel(const D* __restrict__ x, int64_t n_rows, int K,
                                                               int pitch, int8_t* __restrict__ q,
                                                               float* __restrict__ scale) {
  __shared__ uint32_t box[2 * 16];
  int phase = 0;
  for (int64_t row = blockIdx.x; row < n_rows; row += gridDim.x) {
    const D* xr = x + row * K;
    uint32_t top = 0;
    for (int j = threadIdx.x; j < K; j += 1024) top = max_bits(top, __float_as_uint((float)xr[j]) & 0x7fffffffu);
    const RowScale rs = row_scale(row_max_bits<1024, 1024>(top, box, phase));
    if (threadIdx.x == 0) scale[row] = rs.scale;
    for (int j = threadIdx.x * 8; j < pitch; j += 8192) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = j + e < K ? (float)xr[j + e] : 0.f;
      *reinterpret_cast<uint2*>(q + row * pitch + j) = quant8(v, rs);
    }
  }
}

// Gradients of the norm step.  With xh = x' / r, w = gamma dn and mean over a row:
//   d  = dx' + (w - xh mean(w xh)) / r         gradient at x' (its rounding passes it on)
//   dx = res_scale d,  e = block_scale d
//   dgamma += dn xh
//   with yh = y / r_post (or y), b = yh gamma_post, f = gate e, v = gamma_post f:
//   dgate += e b (over the tokens of a gate row),  dgamma_post += f yh
//   dy = (v - yh mean(v yh)) / r_post, or f without a block norm
// A workgroup takes `chunk` consecutive rows and keeps its column sums in
// registers.  Without gates, or where a gate row spans several workgroups, it
// ends with one fp32 partial row per sum; where gate rows are shorter than a
// chunk the chunk holds whole gate rows and writes each dgate row itself; a
// gate row per token needs no sum.
// col_sums_kernel adds the partial rows, in their order: no atomics.
// Bound by HBM: the next row is loaded before the present one is worked on, as
// it lies in memory (bf16 stays packed); the gains are read from LDS.  32768 x
// 4096 bf16 with both norms and gates 0.314 ms, 5.1 TB/s (0.553 without the row
// ahead and with the gains from L2).  1024 lanes (hidden past 8192) have 128
// registers each: no row ahead, and with y 81 to 166 of them spill: 8192 x 16384
// bf16 0.627 ms, 2.6 TB/s (without y 0.250 ms, 5.4 TB/s).
// Y: y is read (a block norm, or dgate is wanted).
template <typename R, typename D, int NT, int CH, bool Y, bool S>
__global__ __launch_bounds__(wg_of(NT), NT <= 512 ? 2 : 4) void block_norm_backward_kernel(const NormGradParams p) {
  constexpr int WG = wg_of(NT), NR = WG / NT;
  constexpr bool SPLIT = sizeof(R) == 4 || sizeof(D) == 4;
  constexpr int CMAX = NT * CH * 8;
  __shared__ __attribute__((aligned(16))) float gains[(Y ? 2 : 1) * CMAX];   // gamma, then gamma_post
  __shared__ uint32_t box[2 * (WG / 64)];
  __shared__ float cols[NR > 1 ? NR * NT * 8 : 1];
  int phase = 0;
  const Lane<NT, SPLIT> ln{(int)threadIdx.x % NT};
  const int sub = threadIdx.x / NT, C = p.C;
  const float inv_c = 1.f / (float)C;
  const bool post = Y && p.gamma_post != nullptr;
  float acc_g[CH][8], acc_p[Y ? CH : 1][8], acc_t[Y ? CH : 1][8];   // dgamma, dgamma_post, dgate
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc_g[c][e] = 0.f;
      if constexpr (Y) acc_p[c][e] = acc_t[c][e] = 0.f;
    }

  // sum of acc over the NR rows a workgroup holds side by side, chunk by chunk;
  // the lanes of sub-row 0 get it and hand it to `put`
  auto fold = [&](float (&acc)[CH][8], auto put) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (NR > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) cols[e * WG + threadIdx.x] = acc[c][e];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int i = 1; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[c][e] += cols[e * WG + i * NT + threadIdx.x];
        }
      }
      if (sub == 0) put(c, acc[c]);
    }
  };

  // a row as it lies in memory
  struct Row {
    Raw8<R, SPLIT> x[CH], dx[CH];
    Raw8<D, SPLIT> dn[CH], y[Y ? CH : 1], gate[CH];
    float r, r_post;
  };
  auto load = [&](Row& a, int64_t row, bool live) __attribute__((always_inline)) {
    const int64_t base = row * C;
    a.r = live && p.dn ? p.r[row] : 0.f;
    a.r_post = live && post ? p.r_post[row] : 1.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      a.x[c].template load<S>(static_cast<const R*>(p.x_out) + base, ln, c, C, live && p.dn);
      a.dn[c].template load<S>(static_cast<const D*>(p.dn) + base, ln, c, C, live && p.dn);
      a.dx[c].template load<S>(static_cast<const R*>(p.dx_out) + base, ln, c, C, live && p.dx_out);
      if constexpr (Y) a.y[c].template load<S>(static_cast<const D*>(p.y) + base, ln, c, C, live);
    }
    const bool gated = p.gate && live;
    const int64_t gbase = gated ? (int64_t)((uint32_t)row / (uint32_t)p.gate_tokens) * C : 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) a.gate[c].template load<false>(static_cast<const D*>(p.gate) + gbase, ln, c, C, gated);
  };
  // rows of this workgroup: chunk `i` of the gate row group it belongs to
  const int64_t group = blockIdx.x / p.spans, i = blockIdx.x % p.spans;
  const int64_t beg = group * p.group_rows + i * p.chunk;
  const int64_t end = min(min(beg + p.chunk, (group + 1) * p.group_rows), p.T);

  Row cur;
  int64_t row0 = beg, seg = beg;                          // segment: the rows up to the next write of dgate
  if (beg < end) load(cur, beg + sub, beg + sub < min(beg + p.flush_rows, end));
  for (int j = threadIdx.x * 4; j < C; j += WG * 4) {
    if (p.gamma) *reinterpret_cast<float4*>(gains + j) = *reinterpret_cast<const float4*>(p.gamma + j);
    if constexpr (Y)
      if (post) *reinterpret_cast<float4*>(gains + CMAX + j) = *reinterpret_cast<const float4*>(p.gamma_post + j);
  }
  __syncthreads();
  while (row0 < end) {
    const int64_t seg_end = min(seg + p.flush_rows, end);
    int64_t next = row0 + NR, next_seg = seg;
    if (next >= seg_end) next = next_seg = seg_end;
    Row ahead;
    auto load_ahead = [&]() __attribute__((always_inline)) {
      if (next < end) load(ahead, next + sub, next + sub < min(next_seg + p.flush_rows, end));
    };
    if constexpr (NT < 1024) load_ahead();                // no room in 1024 lanes

    const int64_t row = row0 + sub;
    const bool live = row < seg_end;
    const int64_t base = row * C;
    const float inv = p.dn && live ? inv_or_zero(cur.r) : 0.f;
    const float invp = post && live ? inv_or_zero(cur.r_post) : 1.f;
    float d[CH][8];
    float s = 0.f, m = 0.f;
    if (p.dn) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float x[8], w[8], g[8];
        cur.x[c].get(x);
        cur.dn[c].get(w);
        load_gain(gains, ln, c, p.gamma ? C : 0, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = w[e] * (x[e] * inv);
          acc_g[c][e] += t;
          s = fmaf(t, g[e], s);
        }
      }
      m = row_sum<NT, WG>(s, box, phase) * inv_c;
    }
    s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float v[8];
      cur.dx[c].get(d[c]);
      if (p.dn) {
        float x[8], w[8], g[8];
        cur.x[c].get(x);
        cur.dn[c].get(w);
        load_gain(gains, ln, c, p.gamma ? C : 0, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[c][e] = fmaf(fmaf(-(x[e] * inv), m, w[e] * g[e]), inv, d[c][e]);
      }
      if (p.dx) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = p.res_scale * d[c][e];
        if (live) store8<S>(static_cast<R*>(p.dx) + base, ln, c, C, v);
      }
      if (!p.block) continue;
      float g[8];
      cur.gate[c].get(g);
      if (!p.gate) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.f;
      }
      if constexpr (Y) {
        float y[8], gp[8];
        cur.y[c].get(y);
        load_gain(gains + CMAX, ln, c, post ? C : 0, gp);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] *= invp;
          d[c][e] *= p.block_scale;
          v[e] = d[c][e] * (y[e] * gp[e]);
          acc_t[c][e] += v[e];
          d[c][e] *= g[e];
          acc_p[c][e] = fmaf(d[c][e], y[e], acc_p[c][e]);
          d[c][e] *= gp[e];
          s = fmaf(d[c][e], y[e], s);
        }
        if (p.gate_each && live) store8<S>(static_cast<D*>(p.dgate) + base, ln, c, C, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[c][e] *= p.block_scale * g[e];
      }
    }
    if (p.block) {
      m = 0.f;
      if (post) m = row_sum<NT, WG>(s, box, phase) * inv_c;
      if (p.dy) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if constexpr (Y) {
            float y[8];
            cur.y[c].get(y);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              // without a block norm dy does not depend on y (0 y is not 0 for a NaN); a branch around the
              // loop spills more: 4096 x 16384 fp32 728 us against 644
              d[c][e] = fmaf(post ? -(y[e] * invp) : 0.f, m, d[c][e]) * invp;
          }
          if (live) store8<S>(static_cast<D*>(p.dy) + base, ln, c, C, d[c]);
        }
      }
    }
    if constexpr (Y) {
      if (next_seg != seg && p.dgate && !p.part_t && !p.gate_each) {
        const int64_t gate_row = seg / p.gate_tokens;
        fold(acc_t, [&](int c, const float (&v)[8]) { store8<false>(static_cast<D*>(p.dgate) + gate_row * C, ln, c, C, v); });
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc_t[c][e] = 0.f;
      }
    }
    if constexpr (NT == 1024) load_ahead();
    row0 = next;
    seg = next_seg;
    cur = ahead;
  }
  const int64_t part = (int64_t)blockIdx.x * C;
  if constexpr (Y) {
    if (p.part_t) fold(acc_t, [&](int c, const float (&v)[8]) { store8<false>(p.part_t + part, ln, c, C, v); });
    if (p.part_p) fold(acc_p, [&](int c, const float (&v)[8]) { store8<false>(p.part_p + part, ln, c, C, v); });
  }
  if (p.part_g) fold(acc_g, [&](int c, const float (&v)[8]) { store8<false>(p.part_g + part, ln, c, C, v); });
}

// Column sums of partial rows, up to three sets in one launch: blockIdx.y 0 is
// dgamma, 1 dgamma_post (each over all `parts` rows), 2 + g row g of dgate (over
// its `spans` rows).  A workgroup has 32 columns x 32 row lanes, 4 columns a
// lane and 8 rows in flight; the lanes' sums are added in a fixed tree.  Bound by
// latency: 512 rows x 1024 columns 4.7 us, x 4096 with all three sets 5.6 us (10
// with 1024 lanes and a tree in LDS).
struct ColSums {
  const float *part_g, *part_p, *part_t;
  float *dgamma, *dgamma_post;
  void* dgate;
  int parts, spans, C, bf16;
};
__global__ __launch_bounds__(256) void col_sums_kernel(const ColSums a) {
  __shared__ f32x4v box[4][8];
  const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3, w = threadIdx.x >> 6, which = blockIdx.y;
  const int c = blockIdx.x * 32 + cx * 4;
  const float* part = which == 0 ? a.part_g : (which == 1 ? a.part_p : a.part_t);
  if (!part) return;
  const int n = which < 2 ? a.parts : a.spans;
  part += (which < 2 ? 0 : (int64_t)(which - 2) * a.spans * a.C) + c;
  f32x4v s = {0.f, 0.f, 0.f, 0.f};
  if (c < a.C)
    for (int i0 = ry; i0 < n; i0 += 256) {
      f32x4v v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        v[u] = f32x4v{0.f, 0.f, 0.f, 0.f};
        if (i0 + 32 * u < n) v[u] = *reinterpret_cast<const f32x4v*>(part + (int64_t)(i0 + 32 * u) * a.C);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v[u][e];
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s[e] += __shfl_xor(s[e], 8);
    s[e] += __shfl_xor(s[e], 16);
    s[e] += __shfl_xor(s[e], 32);
  }
  if ((threadIdx.x & 63) < 8) box[w][cx] = s;
  __syncthreads();
  if (threadIdx.x >= 8 || c >= a.C) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = (box[0][cx][e] + box[1][cx][e]) + (box[2][cx][e] + box[3][cx][e]);
  if (which >= 2 && a.bf16)
    *reinterpret_cast<uint2*>(static_cast<__bf16*>(a.dgate) + (int64_t)(which - 2) * a.C + c) =
        make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  else
    *reinterpret_cast<f32x4v*>((which == 0 ? a.dgamma : which == 1 ? a.dgamma_post
                                : static_cast<float*>(a.dgate) + (int64_t)(which - 2) * a.C) + c) = s;
}

// Whether a call that reads and writes so many bytes passes the caches by: more
// than the 256 MB behind the L2, so that nothing of it would be found there.
// 8-bit rows of 65536 x 1536 bf16 (302 MB): 53 us (75 through the caches); a norm
// step of 75 MB whose inputs were in the cache: 22 us (17 through it).
bool streams(int64_t bytes) { return bytes > (int64_t)256 << 20; }

// rows of the grid: at most `per_cu` workgroups on each of the 256 CUs
int row_grid(int64_t T, int nr, int per_cu) {
  const int64_t need = (T + nr - 1) / nr;
  return (int)(need < 256 * per_cu ? need : 256 * per_cu);
}

template <typename F>
void by_flags(bool a, bool b, F f) {
  if (a) b ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  else b ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}
template <typename R, typename D, int NT, int CH>
hipError_t launch_norm_t(const NormParams& p, bool stream, hipStream_t st) {
  constexpr int WG = wg_of(NT);
  // a stream to two fp tensors runs best with 8 waves a CU: 65536 x 4096 bf16 375 us
  // (425 with 32, 398 with 12, 542 with 4); 8-bit output and short calls with 32
  const int per_cu = stream && !p.q ? std::max(1, 512 / WG) : 2048 / WG;
  by_flags(p.q != nullptr, stream, [&](auto q8, auto s) {
    hipLaunchKernelGGL((block_norm_kernel<R, D, NT, CH, decltype(q8)::value, decltype(s)::value>),
                       dim3(row_grid(p.T, WG / NT, per_cu)), dim3(WG), 0, st, p);
  });
  return hipGetLastError();
}
template <typename R, typename D, int NT, int CH>
hipError_t launch_norm_grad_t(const NormGradParams& p, bool stream, hipStream_t st) {
  by_flags(p.y != nullptr, stream, [&](auto y, auto s) {
    hipLaunchKernelGGL((block_norm_backward_kernel<R, D, NT, CH, decltype(y)::value, decltype(s)::value>),
                       dim3((unsigned)p.n_wg), dim3(wg_of(NT)), 0, st, p);
  });
  return hipGetLastError();
}

// NT lanes x CH chunks of 8 that hold a row of C elements
template <typename F>
hipError_t by_width(int C, F f) {
  using std::integral_constant;
  if (C <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (C <= 1024) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (C <= 2048) return f(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  if (C <= 4096) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (C <= 8192) return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}
// the same for the 8-bit rows, which need few registers: one wave up to 2048
template <typename F>
hipError_t by_quant_width(int C, F f) {
  using std::integral_constant;
  if (C <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (C <= 1024) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (C <= 1536) return f(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  if (C <= 2048) return f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  if (C <= 4096) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (C <= 8192) return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  return f(integral_constant<int, 512>{}, integral_constant<int, 4>{});
}
template <typename F>
hipError_t by_types(int res_bf16, int io_bf16, F f) {
  if (res_bf16) return io_bf16 ? f((__bf16*)0, (__bf16*)0) : f((__bf16*)0, (float*)0);
  return io_bf16 ? f((float*)0, (__bf16*)0) : f((float*)0, (float*)0);
}

}  // namespace

hipError_t launch_block_norm(const NormParams& p, int res_bf16, int io_bf16, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  const int rs = res_bf16 ? 2 : 4, io = io_bf16 ? 2 : 4;
  const bool stream = streams(p.T * p.C * (rs + (p.y ? rs + io : 0) + (p.q ? 1 : p.n ? io : 0)));
  return by_types(res_bf16, io_bf16, [&](auto r, auto d) {
    return by_width(p.C, [&](auto nt, auto ch) {
      return launch_norm_t<std::remove_pointer_t<decltype(r)>, std::remove_pointer_t<decltype(d)>,
                           decltype(nt)::value, decltype(ch)::value>(p, stream, st);
    });
  });
}

// Workgroups and rows of a backward pass (see block_norm_backward_kernel).
NormGradGeometry norm_grad_geometry(int64_t T, int C, int64_t gate_tokens) {
  NormGradGeometry g{};
  const int nt = C <= 1024 ? 64 : (C <= 2048 ? 128 : (C <= 4096 ? 256 : (C <= 8192 ? 512 : 1024)));
  const int nr = wg_of(nt) / nt;
  const int64_t most = nt <= 256 ? 512 : 256;      // workgroups at once: registers leave 8 waves a CU (16 for 1024)
  int64_t rows = std::max<int64_t>(1, (T + most - 1) / most);
  rows = (rows + nr - 1) / nr * nr;
  if (gate_tokens <= 0) {                          // no gate: one chunk after the other
    g.chunk = g.group_rows = g.flush_rows = rows;
    g.spans = 1;
  } else if (gate_tokens == 1) {                   // a gate row per token: written with the token
    g.chunk = g.group_rows = g.flush_rows = rows;
    g.spans = 1;
    g.gate_each = 1;
  } else if (gate_tokens <= rows) {                // whole gate rows in a chunk
    g.chunk = g.group_rows = rows / gate_tokens * gate_tokens;
    g.flush_rows = gate_tokens;
    g.spans = 1;
  } else {                                         // a gate row over `spans` chunks
    g.spans = (int)((gate_tokens + rows - 1) / rows);
    g.chunk = (gate_tokens + g.spans - 1) / g.spans;
    g.flush_rows = g.chunk;
    g.group_rows = gate_tokens;
    g.gate_parts = 1;
  }
  const int64_t groups = (T + g.group_rows - 1) / g.group_rows;
  g.n_wg = groups * g.spans;
  return g;
}

hipError_t launch_block_norm_backward(const NormGradParams& p, int res_bf16, int io_bf16, float* dgamma,
                                      float* dgamma_post, hipStream_t st) {
  const int rs = res_bf16 ? 2 : 4, io = io_bf16 ? 2 : 4;
  const bool stream = streams(p.T * p.C * ((p.dn ? rs + io : 0) + (p.dx_out ? rs : 0) + (p.y ? io : 0) + (p.dx ? rs : 0) +
                                  (p.dy ? io : 0) + (p.gate_each ? io : 0)));
  hipError_t e = p.n_wg == 0 ? hipSuccess : by_types(res_bf16, io_bf16, [&](auto r, auto d) {
    return by_width(p.C, [&](auto nt, auto ch) {
      return launch_norm_grad_t<std::remove_pointer_t<decltype(r)>, std::remove_pointer_t<decltype(d)>,
                                decltype(nt)::value, decltype(ch)::value>(p, stream, st);
    });
  });
  if (e == hipSuccess && (p.part_g || p.part_p || p.part_t)) {
    const ColSums a{p.part_g, p.part_p, p.part_t, dgamma, dgamma_post, p.dgate, (int)p.n_wg, p.spans, p.C, io_bf16};
    const unsigned sets = p.part_t ? 2 + (unsigned)(p.n_wg / p.spans) : 2;
    hipLaunchKernelGGL(col_sums_kernel, dim3((p.C + 31) / 32, sets), dim3(256), 0, st, a);
    e = hipGetLastError();
  }
  return e;
}

namespace {
template <typename D>
hipError_t launch_quant_t(const D* x, int64_t n, int K, int pitch, int8_t* q, float* scale, hipStream_t st) {
  if (pitch > 16384) {
    hipLaunchKernelGGL((quant_long_rows_kernel<D>), dim3(row_grid(n, 1, 2)), dim3(1024), 0, st, x, n, K, pitch, q, scale);
    return hipGetLastError();
  }
  const bool vec = K % 8 == 0;
  const bool stream = vec && streams(n * ((int64_t)K * sizeof(D) + pitch));
  return by_quant_width(pitch, [&](auto nt, auto ch) {
    constexpr int NT = decltype(nt)::value, CH = decltype(ch)::value, WG = wg_of(NT);
    const dim3 grid(row_grid(n, WG / NT, 2048 / WG));
    if (stream) hipLaunchKernelGGL((quant_rows_kernel<D, NT, CH, true, true>), grid, dim3(WG), 0, st, x, n, K, pitch, q, scale);
    else if (vec) hipLaunchKernelGGL((quant_rows_kernel<D, NT, CH, true, false>), grid, dim3(WG), 0, st, x, n, K, pitch, q, scale);
    else hipLaunchKernelGGL((quant_rows_kernel<D, NT, CH, false, false>), grid, dim3(WG), 0, st, x, n, K, pitch, q, scale);
    return hipGetLastError();
  });
}
}  // namespace

hipError_t launch_quant_rows(const void* x, int64_t n, int K, int pitch, int x_bf16, int8_t* q, float* scale,
                             hipStream_t st) {
  if (n == 0) return hipSuccess;
  return x_bf16 ? launch_quant_t(static_cast<const __bf16*>(x), n, K, pitch, q, scale, st)
                : launch_quant_t(static_cast<const float*>(x), n, K, pitch, q, scale, st);
}

}  // namespace hna
