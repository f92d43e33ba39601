// Attention of one new token a sequence over a paged cache, split over the cache's length and joined.
#include "paged_common.hpp"

namespace tc {
namespace dev {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = 4;
constexpr int kTile = 32;                       // cache rows a wave takes at a time
constexpr int kStep = kTile * kAttnWaves;       // and a workgroup
constexpr int kMaxSplit = 2048;                 // rows a workgroup takes at most
constexpr float kInf = __builtin_inff();

// D = A B + C on 16 x 16 tiles with a contraction of 32.  Lane l (r = l % 16, g = l / 16) holds row r
// of A and column r of B at contraction indices 8 g .. 8 g + 7, and column r of C and D at rows 4 g .. 4 g + 3.
template <bool BF16>
__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two fp32 values to two of the 16-bit type, nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (BF16) {
    bf16x2 v;
    v[0] = __bf16(x);
    v[1] = __bf16(y);
    return __builtin_bit_cast(uint32_t, v);
  } else {
    f16x2 v;
    v[0] = _Float16(x);
    v[1] = _Float16(y);
    return __builtin_bit_cast(uint32_t, v);
  }
}
template <bool BF16>
__device__ __forceinline__ float low_half(uint32_t v) {
  if constexpr (BF16) return __builtin_bit_cast(float, v << 16);
  return float(__builtin_bit_cast(f16x2, v)[0]);
}
template <bool BF16>
__device__ __forceinline__ float high_half(uint32_t v) {
  if constexpr (BF16) return __builtin_bit_cast(float, v & 0xffff0000u);
  return float(__builtin_bit_cast(f16x2, v)[1]);
}

// Two e4m3 codes (the low or high half of w) to two values of the 16-bit type: exact in both.
template <bool BF16, bool HIGH>
__device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
  if constexpr (BF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}

// The maximum as the exponents' reference, kept finite: exp2(x - reference) is then 0 for x = -infinity and
// infinite for x = +infinity, so a row of nothing sums to 0 and an infinite logit to infinity (its lse; out,
// infinity over infinity, is NaN).
__device__ __forceinline__ float finite(float top) {
  return __builtin_amdgcn_fmed3f(top, -3.4028234664e38f, 3.4028234664e38f);
}

// One workgroup: up to 16 * HT query heads of one cache head over `split` rows of one sequence.  Its four
// waves take tiles of 32 rows in turn, each with its own running maximum, sum and output (one pass
// over the cache), and meet once at the end.  A wave needs neither LDS nor a barrier in its loop:
//
//   S^T = K Q^T    rows of A are cache rows: lane (r, g) loads 16 bytes of row r straight into A's
//                  layout; Q^T stays in registers.
//   O^T = V^T P^T  S^T leaves lane (r, g) with head r and rows 4 g .. 4 g + 3 of each 16-row half, which is
//                  B's layout if the contraction index 8 g + j stands for row 4 g + j of the first half
//                  (j < 4) or 4 g + j - 4 of the second: the softmax's output feeds the product as it is.
//                  For V^T lane (r, g) loads, of those eight rows, the same DP / 16 neighbouring
//                  elements (16 lanes: a whole row) and regroups them by byte permutes.
//
// P is held as the sum of two 16-bit values (its rounding and the rest), two products each: the matrix
// cores are idle nine cycles in ten here, and out is then as exact as fp32 sums of fp32 weights.
// 8-bit rows become 16-bit values in registers (exactly); the key's scale multiplies its row's
// logits, the value's its row's weights.
//
// DP: head_dim rounded up to 64, 128 or 256 (elements past head_dim are zeros).  PAGE16: pages of a multiple of 16
// rows, so that a 16-row half lies on one page and its address is found once a wave; otherwise, and
// for a split's last rows and splits with a missing page, each lane finds its rows' addresses itself.
//
// Bound: HBM (a cache row is read once for all heads of its group).
template <bool BF16, bool E4M3, int DP, int HT, bool PAGE16>
struct Attend {
  static constexpr bool VBF = BF16 || E4M3;       // type of the second product
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int KS = DP / 32;              // contraction steps of the first product
  static constexpr int KC = DP * EB / 64;         // 16-byte chunks a lane loads of a key row
  static constexpr int VF = DP / 16;              // elements a lane loads of a value row: tiles of O^T
  static constexpr int VB = VF * EB;              // their bytes: 4, 8, 16 or 32
  static constexpr int VW = VB / 4;

  // The element of Q that contraction index (step s, group g, j) stands for.
  static __device__ __forceinline__ int q_element(int s, int g, int j) {
    if constexpr (E4M3) return ((s >> 1) * 4 + g) * 16 + (s & 1) * 8 + j;
    return s * 32 + g * 8 + j;
  }
  // The element of row r of tile f of O^T (VF > 8: two halves, so that a load covers whole lines).
  static __device__ __forceinline__ int v_element(int r, int f) {
    if constexpr (VB == 32) return (f >> 3) * (DP / 2) + r * 8 + (f & 7);
    return r * VF + f;
  }

  static __device__ void run(const AttentionArgs& a, int b, int h, int gt, int sp);
};

// Dwords of a value row at lane r: VB bytes, in 16-byte pieces DP / 2 elements apart.
template <int VB>
__device__ __forceinline__ void load_v(const unsigned char* p, int half_bytes, bool first, bool second, uint32_t* w) {
  if constexpr (VB == 32) {
    if (first) load_words<16>(p, w);
    if (second) load_words<16>(p + half_bytes, w + 4);
  } else {
    if (first) load_words<VB>(p, w);
  }
}

template <bool BF16, bool E4M3, int DP, int HT, bool PAGE16>
__device__ __forceinline__ void Attend<BF16, E4M3, DP, HT, PAGE16>::run(const AttentionArgs& a, int b, int h, int gt,
                                                                      int sp) {
  __shared__ int pages[kMaxSplit + 2];
  __shared__ float merge_ml[kAttnWaves][2][16];
  __shared__ float merge_o[kAttnWaves][16][DP + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n = paged_len(a.lens, b, a.max_len);
  const int t0 = sp * a.split;
  if (t0 >= n && sp > 0) return;
  const int t1 = t0 + a.split < n ? t0 + a.split : n;  // this workgroup's rows [t0, t1)
  const PagedPool& p = a.pool;
  const int g0 = gt * 16 * HT;  // its first head in the group

  // the split's pages, -1 for none
  const uint32_t c0 = udiv(uint32_t(t0), p.div);
  bool missing = false;
  if (t1 > t0) {
    const uint32_t cn = udiv(uint32_t(t1 - 1), p.div) - c0 + 1;
    for (uint32_t i = tid; i < cn; i += kAttnThreads) {
      const int page = paged_page(a.table, p, b, c0 + i);
      pages[i] = page;
      missing = missing || page < 0;
    }
  }

  // Q^T: column r is head g0 + 16 ht + r
  u32x4 q[HT][KS];
#pragma unroll
  for (int ht = 0; ht < HT; ++ht) {
    const int head = g0 + 16 * ht + r;
    const unsigned char* row = a.q + b * a.qb + (int64_t(h) * a.group + head) * a.qh;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 v = {};
      const int d = q_element(s, g, 0);
      if (head < a.group && d < a.head_dim) {
        const uint16_t* e = reinterpret_cast<const uint16_t*>(row) + d;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = uint32_t(e[2 * i]) | uint32_t(e[2 * i + 1]) << 16;
      }
      q[ht][s] = v;
    }
  }
  missing = __syncthreads_or(missing);

  f32x4 o[HT][VF];
  float m[HT], l[HT];  // of head r: the maximum over the wave's rows, the sum over the lane's
#pragma unroll
  for (int ht = 0; ht < HT; ++ht) {
    m[ht] = -kInf;
    l[ht] = 0.0f;
#pragma unroll
    for (int f = 0; f < VF; ++f) o[ht][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const unsigned char* kbase = p.k + h * p.kh;
  const unsigned char* vbase = p.v + h * p.vh;
  const int ke = a.head_dim * EB / 16;  // 16-byte chunks of a key row
  const int v0 = v_element(r, 0);
  const bool vok0 = v0 < a.head_dim, vok1 = VB == 32 && v0 + DP / 2 < a.head_dim;

  for (int t = t0 + wave * kTile; t < t1; t += kStep) {
    u32x4 kr[2][KC];
    uint32_t vr[8][VW];
    float ksc = 1.0f, vsc = 1.0f;  // 8-bit rows: lane i holds the scales of the tile's row i % 32
    bool valid[2][4];              // rows 4 g + j of each half
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < KC; ++c) kr[u][c] = u32x4{};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < VW; ++i) vr[j][i] = 0;
    const bool whole = PAGE16 && !missing && t + kTile <= t1;
    if (whole) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t at = uint32_t(t + 16 * u), c = udiv(at, p.div);
        const int page = __builtin_amdgcn_readfirstlane(pages[c - c0]);
        const uint32_t row = at - c * p.div.d;
        const unsigned char* kp = kbase + page * p.kp + (row + r) * p.kr + 16 * g;
        const unsigned char* vp = vbase + page * p.vp + (row + 4 * g) * p.vr + v0 * EB;
#pragma unroll
        for (int i = 0; i < KC; ++i)
          if (4 * i + g < ke) load_words<16>(kp + 64 * i, reinterpret_cast<uint32_t*>(&kr[u][i]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          load_v<VB>(vp + j * p.vr, DP / 2 * EB, vok0, vok1, vr[4 * u + j]);
          valid[u][j] = true;
        }
        if (E4M3 && ((lane >> 4) & 1) == u) {
          ksc = p.ks[page * p.ksp + (row + r) * p.ksr + h * p.ksh];
          vsc = p.vs[page * p.vsp + (row + r) * p.vsr + h * p.vsh];
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = t + 16 * u + r;
        if (at < t1) {
          const uint32_t c = udiv(uint32_t(at), p.div);
          const int page = pages[c - c0];
          if (page >= 0) {
            const uint32_t row = uint32_t(at) - c * p.div.d;
            const unsigned char* kp = kbase + page * p.kp + row * p.kr + 16 * g;
#pragma unroll
            for (int i = 0; i < KC; ++i)
              if (4 * i + g < ke) load_words<16>(kp + 64 * i, reinterpret_cast<uint32_t*>(&kr[u][i]));
            if (E4M3 && ((lane >> 4) & 1) == u) {
              ksc = p.ks[page * p.ksp + row * p.ksr + h * p.ksh];
              vsc = p.vs[page * p.vsp + row * p.vsr + h * p.vsh];
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int av = t + 16 * u + 4 * g + j;
          valid[u][j] = false;
          if (av < t1) {
            const uint32_t c = udiv(uint32_t(av), p.div);
            const int page = pages[c - c0];
            if (page >= 0) {
              const uint32_t row = uint32_t(av) - c * p.div.d;
              load_v<VB>(vbase + page * p.vp + row * p.vr + v0 * EB, DP / 2 * EB, vok0, vok1, vr[4 * u + j]);
              valid[u][j] = true;
            }
          }
        }
      }
    }

    // S^T, scaled into base-2 logits; rows that do not exist are -infinity
    float s[HT][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 acc[HT];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) acc[ht] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        u32x4 x;
        if constexpr (E4M3) {
          const u32x4& w = kr[u][k >> 1];
          const uint32_t w0 = w[(k & 1) * 2], w1 = w[(k & 1) * 2 + 1];
          x = u32x4{from_e4m3<BF16, false>(w0), from_e4m3<BF16, true>(w0), from_e4m3<BF16, false>(w1),
                    from_e4m3<BF16, true>(w1)};
        } else {
          x = kr[u][k];
        }
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) acc[ht] = mfma<BF16>(x, q[ht][k], acc[ht]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f = a.scale_log2e;
        if constexpr (E4M3) f *= __shfl(ksc, 16 * u + 4 * g + j, 64);
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) s[ht][u][j] = valid[u][j] ? acc[ht][j] * f : -kInf;
      }
    }
    float vs[2][4];
    if constexpr (E4M3) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) vs[u][j] = __shfl(vsc, 16 * u + 4 * g + j, 64);
    }
    if (a.logits) {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        const int head = g0 + 16 * ht + r;
        if (head < a.group) {
          float* row = a.logits + ((int64_t(b) * a.heads + h) * a.group + head) * a.logit_row + t + 4 * g;
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<f32x4*>(row + 16 * u) = f32x4{s[ht][u][0], s[ht][u][1], s[ht][u][2], s[ht][u][3]};
        }
      }
    }

    // online softmax, and P^T in B's layout as two 16-bit parts
    u32x4 hi[HT], lo[HT];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      float top = m[ht];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, s[ht][u][j]);
      top = __builtin_fmaxf(top, lane_xor<16>(top));
      top = __builtin_fmaxf(top, lane_xor<32>(top));
      const float ref = finite(top);
      if (__ballot(top > m[ht])) {
        const float shrink = __builtin_amdgcn_exp2f(m[ht] - ref);
        l[ht] *= shrink;
#pragma unroll
        for (int f = 0; f < VF; ++f) o[ht][f] *= shrink;
        m[ht] = top;
      }
      float x[8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float e = __builtin_amdgcn_exp2f(s[ht][u][j] - ref);
          l[ht] += e;
          if constexpr (E4M3) e = valid[u][j] ? e * vs[u][j] : 0.0f;
          x[4 * u + j] = e;
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[ht][i] = pack2<VBF>(x[2 * i], x[2 * i + 1]);
        lo[ht][i] = pack2<VBF>(x[2 * i] - low_half<VBF>(hi[ht][i]), x[2 * i + 1] - high_half<VBF>(hi[ht][i]));
      }
    }

    // O^T += V^T P^T
#pragma unroll
    for (int f = 0; f < VF; ++f) {
      u32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E4M3) {
          // bytes f of rows 2 i and 2 i + 1, side by side
          const uint32_t pair = perm(vr[2 * i + 1][f >> 2], vr[2 * i][f >> 2],
                                     uint32_t((f & 3) | ((f & 3) + 4) << 8));
          x[i] = from_e4m3<true, false>(pair);
        } else {
          x[i] = perm(vr[2 * i + 1][f >> 1], vr[2 * i][f >> 1], f & 1 ? 0x07060302u : 0x05040100u);
        }
      }
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        o[ht][f] = mfma<VBF>(x, hi[ht], o[ht][f]);
        o[ht][f] = mfma<VBF>(x, lo[ht], o[ht][f]);
      }
    }
  }

  // the four waves' parts of each 16 heads
  const int64_t hq0 = (int64_t(b) * a.heads + h) * a.group;
#pragma unroll
  for (int ht = 0; ht < HT; ++ht) {
    l[ht] += lane_xor<16>(l[ht]);
    l[ht] += lane_xor<32>(l[ht]);
    if (ht > 0) __syncthreads();  // the last heads' parts have been read
    if (g == 0) {
      merge_ml[wave][0][r] = m[ht];
      merge_ml[wave][1][r] = l[ht];
    }
    __syncthreads();
    float top = -kInf;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) top = __builtin_fmaxf(top, merge_ml[w][0][r]);
    const float mine = __builtin_amdgcn_exp2f(m[ht] - finite(top));
#pragma unroll
    for (int f = 0; f < VF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) merge_o[wave][r][v_element(4 * g + i, f)] = o[ht][f][i] * mine;
    __syncthreads();
    const int d0 = tid % (DP / 4) * 4;
    for (int head = tid / (DP / 4); head < 16; head += kAttnThreads / (DP / 4)) {
      const int hg = g0 + 16 * ht + head;
      if (hg >= a.group || d0 >= a.head_dim) continue;
      float mx = -kInf, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) mx = __builtin_fmaxf(mx, merge_ml[w][0][head]);
      const float ref = finite(mx);
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) {
        sum += merge_ml[w][1][head] * __builtin_amdgcn_exp2f(merge_ml[w][0][head] - ref);
        acc += *reinterpret_cast<const f32x4*>(&merge_o[w][head][d0]);
      }
      const int64_t hq = hq0 + hg;
      if (d0 == 0 && a.part_ml) {
        a.part_ml[(hq * a.splits + sp) * 2] = mx;
        a.part_ml[(hq * a.splits + sp) * 2 + 1] = sum;
      }
      if (a.splits > 1) {
        *reinterpret_cast<f32x4*>(a.part_o + (hq * a.splits + sp) * a.head_dim + d0) = acc;
      } else {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint16_t* out = reinterpret_cast<uint16_t*>(a.out + b * a.ob + (int64_t(h) * a.group + hg) * a.oh) + d0;
        const uint32_t w0 = pack2<BF16>(acc[0] * inv, acc[1] * inv), w1 = pack2<BF16>(acc[2] * inv, acc[3] * inv);
        out[0] = uint16_t(w0);
        out[1] = uint16_t(w0 >> 16);
        out[2] = uint16_t(w1);
        out[3] = uint16_t(w1 >> 16);
        if (d0 == 0 && a.lse)
          a.lse[b * a.lb + (int64_t(h) * a.group + hg) * a.lh] = (mx + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
      }
    }
  }
}

// Grid: (split, sequence, cache head), the heads fastest; blockIdx.y: tiles of 16 * HT heads of the group.
template <bool BF16, bool E4M3, int DP, int HT, bool PAGE16>
__global__ __launch_bounds__(kAttnThreads) void paged_attention_kernel(AttentionArgs a, Div32 heads, Div32 batch) {
  const uint32_t x = blockIdx.x, bs = udiv(x, heads), sp = udiv(bs, batch);
  Attend<BF16, E4M3, DP, HT, PAGE16>::run(a, int(bs - sp * batch.d), int(x - bs * heads.d), int(blockIdx.y), int(sp));
}

// The splits of one query head joined: their maxima give each split's factor, the sums and outputs are
// added in a fixed order.  One workgroup a (sequence, query head); lanes of four elements, rounds of splits.
template <bool BF16>
__global__ __launch_bounds__(256) void paged_join_kernel(AttentionArgs a, Div32 q_heads) {
  __shared__ float part[8][kPagedMaxHeadDim];
  __shared__ float sums[8];
  const int hq = int(blockIdx.x), b = int(udiv(blockIdx.x, q_heads)), hh = hq - b * int(q_heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int used = n > 0 ? (n + a.split - 1) / a.split : 0;
  const float* ml = a.part_ml + int64_t(hq) * a.splits * 2;
  const float* po = a.part_o + int64_t(hq) * a.splits * a.head_dim;
  float top = -kInf;
  for (int i = threadIdx.x & 63; i < used; i += 64) top = __builtin_fmaxf(top, ml[2 * i]);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
  const float ref = finite(top);
  const int lane4 = threadIdx.x & 31, grp = threadIdx.x >> 5;
  f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
  float sum = 0.0f;
  for (int i = grp; i < used; i += 8) {
    const float f = __builtin_amdgcn_exp2f(ml[2 * i] - ref);
    sum += ml[2 * i + 1] * f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 4 * lane4 + 128 * k;
      if (d < a.head_dim) acc[k] += *reinterpret_cast<const f32x4*>(po + int64_t(i) * a.head_dim + d) * f;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[grp][4 * lane4 + 128 * k + i] = acc[k][i];
  if (lane4 == 0) sums[grp] = sum;
  __syncthreads();
  const int d = threadIdx.x;
  float total = 0.0f, x = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    total += sums[k];
    x += part[k][d];
  }
  if (d < a.head_dim) {
    x = total == 0.0f ? 0.0f : x * (1.0f / total);
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out + b * a.ob + hh * a.oh) + d;
    *out = uint16_t(pack2<BF16>(x, 0.0f));
  }
  if (d == 0 && a.lse) a.lse[b * a.lb + hh * a.lh] = (top + __builtin_amdgcn_logf(total)) * 0.6931471805599453f;
}

// weights_out[i] = weights[i] + the sum over a cache head's query heads of exp2(logit - lse), lse again
// from the splits.  One workgroup a kWeightRows rows of one (sequence, cache head).
constexpr int kWeightRows = 1024;
__global__ __launch_bounds__(256) void paged_weights_kernel(AttentionArgs a, Div32 heads, Div32 chunks) {
  const uint32_t bh = udiv(blockIdx.x, chunks), chunk = blockIdx.x - bh * chunks.d;
  const int b = int(udiv(bh, heads)), h = int(bh - uint32_t(b) * heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int i0 = int(chunk) * kWeightRows;
  if (i0 >= n) return;
  const int used = (n + a.split - 1) / a.split;
  const float* w = a.weights + b * a.w.sb + h * a.w.sh;
  float* wo = a.weights_out + b * a.wo.sb + h * a.wo.sh;
  float sum[kWeightRows / 256] = {};
  for (int g = 0; g < a.group; ++g) {
    const int64_t hq = int64_t(bh) * a.group + g;
    const float* ml = a.part_ml + hq * a.splits * 2;
    float top = -kInf, total = 0.0f;
    for (int i = threadIdx.x & 63; i < used; i += 64) top = __builtin_fmaxf(top, ml[2 * i]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
    const float ref = finite(top);
    for (int i = threadIdx.x & 63; i < used; i += 64) total += ml[2 * i + 1] * __builtin_amdgcn_exp2f(ml[2 * i] - ref);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d, 64);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const float* x = a.logits + hq * a.logit_row;
#pragma unroll
    for (int k = 0; k < kWeightRows / 256; ++k) {
      const int i = i0 + 256 * k + int(threadIdx.x);
      if (i < n) sum[k] += __builtin_amdgcn_exp2f(x[i] - ref) * inv;
    }
  }
#pragma unroll
  for (int k = 0; k < kWeightRows / 256; ++k) {
    const int i = i0 + 256 * k + int(threadIdx.x);
    if (i < n) wo[i * a.wo.sc] = w[i * a.w.sc] + sum[k];
  }
}

template <bool BF16, bool E4M3, int DP, int HT, bool PAGE16>
void attend(const AttentionArgs& a, hipStream_t s) {
  const uint32_t wgs = uint32_t(a.splits) * uint32_t(a.table.batch) * uint32_t(a.heads);
  hipLaunchKernelGGL((paged_attention_kernel<BF16, E4M3, DP, HT, PAGE16>), dim3(wgs, uint32_t((a.group + 16 * HT - 1) / (16 * HT))),
                     dim3(kAttnThreads), 0, s, a, make_div32(uint32_t(a.heads)), make_div32(uint32_t(a.table.batch)));
}

template <bool BF16, bool E4M3, int DP>
void by_group(const AttentionArgs& a, hipStream_t s) {
  const bool page16 = a.pool.page_size % 16 == 0;
  if (a.group <= 16) return page16 ? attend<BF16, E4M3, DP, 1, true>(a, s) : attend<BF16, E4M3, DP, 1, false>(a, s);
  return page16 ? attend<BF16, E4M3, DP, 2, true>(a, s) : attend<BF16, E4M3, DP, 2, false>(a, s);
}

template <bool BF16, bool E4M3>
void by_dim(const AttentionArgs& a, hipStream_t s) {
  if (a.head_dim <= 64) return by_group<BF16, E4M3, 64>(a, s);
  if (a.head_dim <= 128) return by_group<BF16, E4M3, 128>(a, s);
  return by_group<BF16, E4M3, 256>(a, s);
}

}  // namespace dev

int64_t paged_logit_row(int64_t max_len) { return (max_len + dev::kStep - 1) / dev::kStep * dev::kStep; }

PagedSplit paged_split(int64_t batch, int64_t heads, int64_t group, int64_t max_len) {
  const int64_t pairs = batch * heads * ((group + 31) / 32);
  int64_t rows = 256;
  if (max_len <= rows) return PagedSplit{int32_t(rows), 1};
  while (rows < dev::kMaxSplit && pairs * ((max_len + 2 * rows - 1) / (2 * rows)) >= 1024) rows *= 2;
  return PagedSplit{int32_t(rows), int32_t((max_len + rows - 1) / rows)};
}

int launch_paged_attention(const AttentionArgs& in, int dtype, int cache_dtype, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  AttentionArgs a = in;
  const int64_t pairs = int64_t(a.table.batch) * a.heads;
  if (pairs * a.splits >= int64_t(1) << 31 || (a.group + 15) / 16 > 65535) return TC_E_RANGE;
  const int64_t chunks = (int64_t(a.max_len) + dev::kWeightRows - 1) / dev::kWeightRows;
  if (pairs * chunks >= int64_t(1) << 31) return TC_E_RANGE;
  if (!a.weights_out) a.logits = nullptr;
  if (a.splits == 1 && !a.weights_out) a.part_ml = nullptr;
  const bool bf16 = dtype == TC_BF16, e4m3 = cache_dtype == TC_E4M3;
  if (bf16)
    e4m3 ? dev::by_dim<true, true>(a, s) : dev::by_dim<true, false>(a, s);
  else
    e4m3 ? dev::by_dim<false, true>(a, s) : dev::by_dim<false, false>(a, s);
  const uint32_t hq = uint32_t(pairs) * uint32_t(a.group);
  if (a.splits > 1) {
    const Div32 qh = make_div32(uint32_t(a.heads) * uint32_t(a.group));
    if (bf16)
      hipLaunchKernelGGL(dev::paged_join_kernel<true>, dim3(hq), dim3(256), 0, s, a, qh);
    else
      hipLaunchKernelGGL(dev::paged_join_kernel<false>, dim3(hq), dim3(256), 0, s, a, qh);
  }
  if (a.weights_out && chunks > 0)
    hipLaunchKernelGGL(dev::paged_weights_kernel, dim3(uint32_t(pairs * chunks)), dim3(256), 0, s, a,
                       make_div32(uint32_t(a.heads)), make_div32(uint32_t(chunks)));
  return TC_OK;
}

}  // namespace tc
