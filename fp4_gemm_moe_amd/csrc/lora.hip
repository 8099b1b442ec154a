// Low-rank adapters: v = x A[g]^T by place (shrink), out = base + scale[g] v
// B[g]^T by token (expand), and the gradients: u = dy B[g] (shrink), dx = base +
// scale[g] u A[g] (expand), dA = scale u^T x and dB = scale dy^T v (outer).
#include <atomic>
#include <type_traits>

#include "group_tiles.hpp"
#include "half_internal.hpp"
#include "half_math.hpp"

namespace hq {
namespace {

extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

__device__ __forceinline__ int64_t token_at(const LoraPlan& pl, int place) {
  const int64_t t = pl.row_pair != nullptr ? pl.row_pair[place] : place;
  return t >= 0 && t < pl.m ? t : -1;
}
__device__ __forceinline__ v4i load8(const uint16_t* p) { return *reinterpret_cast<const v4i*>(p); }

// ------------------------------------------------------------------ shrink
constexpr int kShrinkWaves = 8;

// Partial sums of a workgroup: 16 MF places x 16 RF ranks over one slice of K.
// Its waves take blocks of 64 K values in turn, each lane loading its operands
// from memory (w [K, r]: through the wave's share of LDS, read transposed), and
// their sums meet in LDS in the order of the waves.
struct ShrinkArgs {
  LoraPlan pl;
  const uint16_t* z;       // [m, k]
  const uint16_t* w;       // [adapters, r, k]; WT: [adapters, k, r]
  float* out;              // [slices, max_rows, r]
  int k, r, slices;
};

template <bool F16, bool WT, int MF, int RF>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink(ShrinkArgs p) {
  constexpr int W = kShrinkWaves, RN = 16 * RF, PITCH = RN * 2 + 16;
  constexpr int U = WT ? 1 : 2;                     // blocks in flight
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), x = lane & 15, q = lane >> 4;
  const int chunks = (p.r + RN - 1) / RN;
  int id = blockIdx.x;
  const int slice = id % p.slices;
  id /= p.slices;
  const int r0 = id % chunks * RN;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 16 * MF, id / chunks);
  if (t.g < 0) return;
  const uint16_t* zp[MF];
  bool live[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int place = t.row0 + 16 * i + x;
    const int64_t tok = place < t.row_end ? token_at(p.pl, place) : -1;
    live[i] = tok >= 0;
    zp[i] = p.z + (tok >= 0 ? tok : 0) * p.k + 8 * q;
  }
  const uint16_t* wg = p.w + (int64_t)t.g * p.r * p.k;
  const uint16_t* wp[RF];
  if constexpr (!WT) {
#pragma unroll
    for (int j = 0; j < RF; ++j) {
      const int row = r0 + 16 * j + x;
      wp[j] = wg + (int64_t)(row < p.r ? row : p.r - 1) * p.k + 8 * q;
    }
  }
  uint8_t* mine = smem + w * 64 * PITCH;
  v4f acc[MF][RF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < RF; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  const int blocks = (p.k + 63) / 64, last = blocks * (slice + 1) / p.slices;
  for (int b = blocks * slice / p.slices + w * U; b < last; b += W * U) {
    v4i zf[U][2][MF], wf[U][2][RF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = (b + u) * 64;
      const bool on = b + u < last;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = on && k0 + 32 * h + 8 * q < p.k;
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          zf[u][h][i] = v4i{0, 0, 0, 0};
          if (in && live[i]) zf[u][h][i] = load8(zp[i] + k0 + 32 * h);
        }
        if constexpr (!WT) {
#pragma unroll
          for (int j = 0; j < RF; ++j) {
            wf[u][h][j] = v4i{0, 0, 0, 0};
            if (in) wf[u][h][j] = load8(wp[j] + k0 + 32 * h);
          }
        }
      }
      if constexpr (WT) {
        // 64 rows of RN ranks: RN / 8 pieces of 16 bytes a lane
        v4i piece[2 * RF];
#pragma unroll
        for (int e = 0; e < 2 * RF; ++e) {
          const int c = lane + 64 * e, row = c / (2 * RF), col = c % (2 * RF) * 8;
          piece[e] = v4i{0, 0, 0, 0};
          if (k0 + row < p.k && r0 + col < p.r) piece[e] = load8(wg + (int64_t)(k0 + row) * p.r + r0 + col);
        }
#pragma unroll
        for (int e = 0; e < 2 * RF; ++e) {
          const int c = lane + 64 * e, row = c / (2 * RF), col = c % (2 * RF) * 8;
          *reinterpret_cast<v4i*>(mine + row * PITCH + col * 2) = piece[e];
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < RF; ++j) {
            const uint8_t* at = mine + (32 * h + 8 * q + (x >> 2)) * PITCH + (16 * j + 4 * (x & 3)) * 2;
            wf[u][h][j] = join(read_transposed(at), read_transposed(at + 4 * PITCH));
          }
        asm volatile("" ::: "memory");
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int j = 0; j < RF; ++j) acc[i][j] = product16<F16>(wf[u][h][j], zf[u][h][i], acc[i][j]);
  }
  v4f* part = reinterpret_cast<v4f*>(smem);         // [W][MF * RF][64]
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < RF; ++j) part[(w * MF * RF + i * RF + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int f = w; f < MF * RF; f += W) {
    v4f s = part[f * 64 + lane];
#pragma unroll
    for (int e = 1; e < W; ++e) s += part[(e * MF * RF + f) * 64 + lane];
    const int i = f / RF, place = t.row0 + 16 * i + x, rank = r0 + 16 * (f % RF) + 4 * q;
    if (place < t.row_end && rank < p.r && token_at(p.pl, place) >= 0)
      *reinterpret_cast<v4f*>(p.out + ((int64_t)slice * p.pl.max_rows + place) * p.r + rank) = s;
  }
}

// ------------------------------------------------------------------ expand
constexpr int kThreads = 256;

struct ExpandArgs {
  LoraPlan pl;
  const float* v;          // [slices, max_rows, r]
  const uint16_t* w;       // [adapters, n, r]; WT: [adapters, r, n]
  const uint16_t* base;
  uint16_t* out;           // [m, n]
  float* v_out;            // the slices' sums (nullptr: not kept)
  int n, r, slices;
  int chunk;               // columns of a workgroup, a multiple of 256
  int chunks;
  unsigned tiles, rest;    // workgroups of places, of tokens without an adapter
};
constexpr int kRestRows = 64;
constexpr int kWtRanks = 64;             // WT: ranks of w in LDS at a time

// Bytes of LDS: 16 MF places of r values as two 16-bit parts, and their factors; WT:
// a wave's 64 columns of w.
template <bool WT, int MF>
constexpr int expand_smem(int r) {
  return 16 * MF * ((r + 15) / 16 * 64 + 16) + 16 * MF * 4 + (WT ? 4 * kWtRanks * 144 : 0);
}

// Tokens without an adapter: base's row, or zeros.
__device__ __forceinline__ void expand_rest(const ExpandArgs& p, int id) {
  const int c0 = id % p.chunks * p.chunk, c1 = c0 + p.chunk < p.n ? c0 + p.chunk : p.n;
  const int64_t t0 = (int64_t)(id / p.chunks) * kRestRows;
  const int last = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 1, 0).last;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = wave; i < kRestRows; i += 4) {
    const int64_t t = t0 + i;
    if (t >= p.pl.m) break;
    const int64_t place = p.pl.row_map != nullptr ? p.pl.row_map[t] : t;
    if (place >= 0 && place < last) continue;
    for (int c = c0 + lane * 8; c < c1; c += 512)
      *reinterpret_cast<v4i*>(p.out + t * p.n + c) = p.base != nullptr ? load8(p.base + t * p.n + c) : v4i{0, 0, 0, 0};
  }
}

// A workgroup: 16 MF places, `chunk` columns; each wave 64 of every 256.  A place's
// value v scale is kept as hi + lo: 16 ranks' hi and 16 ranks' lo are the 32 K
// values of one matrix product with the ranks' weights twice.  BF16: hi the value
// cut to 8 bits, lo the rest rounded.  FP16: the place's values are first scaled
// by the power of two that takes the largest to [2^14, 2^15), undone in FP32 at
// the end, so that neither part leaves FP16's range.
template <bool F16, bool WT, int MF>
__device__ __forceinline__ void expand_tile(const ExpandArgs& p, int id) {
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), x = lane & 15, q = lane >> 4;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 16 * MF, id / p.chunks);
  if (t.g < 0) return;
  const int chunk_no = id % p.chunks, c0 = chunk_no * p.chunk, c1 = c0 + p.chunk < p.n ? c0 + p.chunk : p.n;
  const int steps = (p.r + 15) / 16, pitch = steps * 64 + 16;
  uint8_t* vt = smem;
  float* fac = reinterpret_cast<float*>(smem + 16 * MF * pitch);
  uint8_t* wt = smem + 16 * MF * (pitch + 4) + w * kWtRanks * 144;
  const float scale = p.pl.scale != nullptr ? p.pl.scale[t.g] : 1.0f;

  // the places' values: 16 threads a place, in pairs of ranks
#pragma unroll 1
  for (int i = tid >> 4; i < 16 * MF; i += 16) {
    const int place = t.row0 + i;
    const bool on = place < t.row_end && token_at(p.pl, place) >= 0;
    auto value = [&](int rank) -> float2 {
      float2 s = make_float2(0.0f, 0.0f);
      if (!on || rank >= p.r) return s;
      const float* src = p.v + (int64_t)place * p.r + rank;
      s = *reinterpret_cast<const float2*>(src);
      for (int e = 1; e < p.slices; ++e) {
        const float2 o = *reinterpret_cast<const float2*>(src + (int64_t)e * p.pl.max_rows * p.r);
        s.x += o.x;
        s.y += o.y;
      }
      return s;
    };
    float f = 1.0f, back = 1.0f;
    if constexpr (F16) {
      uint32_t top = 0;
      for (int rank = 2 * x; rank < p.r; rank += 32) {
        const float2 s = value(rank);
        const uint32_t a = __float_as_uint(s.x * scale) & 0x7fffffffu, b = __float_as_uint(s.y * scale) & 0x7fffffffu;
        top = a > top ? a : top;
        top = b > top ? b : top;
      }
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)top, off, 16);
        top = o > top ? o : top;
      }
      int e = (int)(top >> 23);                                        // biased exponent
      e = e < 15 ? 15 : (e > 254 ? 141 : e);                           // Inf and NaN: unscaled
      f = __uint_as_float((uint32_t)(127 + 141 - e) << 23);
      back = __uint_as_float((uint32_t)(127 - 141 + e) << 23);
    }
    for (int rank = 2 * x; rank < steps * 16; rank += 32) {
      const float2 s = value(rank);
      if (p.v_out != nullptr && chunk_no == 0 && on && rank < p.r)
        *reinterpret_cast<float2*>(p.v_out + (int64_t)place * p.r + rank) = s;
      const float a = s.x * scale, b = s.y * scale;
      uint32_t hi, lo;
      if constexpr (F16) {
        const float fa = a * f, fb = b * f;
        hi = pack_half2<true>(fa, fb);
        const float ha = f16_lo(hi), hb = f16_hi(hi);
        lo = pack_half2<true>(__builtin_fabsf(ha) == INFINITY ? 0.0f : fa - ha, __builtin_fabsf(hb) == INFINITY ? 0.0f : fb - hb);
      } else {
        const float ca = bf16_cut(a), cb = bf16_cut(b);
        hi = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
        if (a != a) hi |= 0x7fc0u;                                       // a NaN whose top bits are an infinity's
        if (b != b) hi |= 0x7fc00000u;
        lo = pack_half2<false>(bf16_rest(a, ca), bf16_rest(b, cb));
      }
      uint8_t* d = vt + i * pitch + (rank >> 4) * 64 + (rank & 15) * 2;
      *reinterpret_cast<uint32_t*>(d) = hi;
      *reinterpret_cast<uint32_t*>(d + 32) = lo;
    }
    if (x == 0) fac[i] = back;
  }
  __syncthreads();

  int64_t tok[MF];
  float back[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int place = t.row0 + 16 * i + x;
    tok[i] = place < t.row_end ? token_at(p.pl, place) : -1;
    back[i] = F16 ? fac[16 * i + x] : 1.0f;
  }
  const uint16_t* wg = p.w + (int64_t)t.g * p.r * p.n;
  for (int n0 = c0 + w * 64; n0 < c1; n0 += 256) {
    // columns of a lane: 32 jp + 8 q .. + 7; a fragment j of a pair has 8 (x / 4) + 4 j + x % 4
    v4i bs[2][MF];
#pragma unroll
    for (int jp = 0; jp < 2; ++jp)
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int col = n0 + 32 * jp + 8 * q;
        bs[jp][i] = v4i{0, 0, 0, 0};
        if (p.base != nullptr && tok[i] >= 0 && col < c1) bs[jp][i] = load8(p.base + tok[i] * p.n + col);
      }
    v4f acc[MF][4];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    const uint16_t* wp[4];
    if constexpr (!WT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = n0 + 32 * (j >> 1) + 8 * (x >> 2) + 4 * (j & 1) + (x & 3);
        wp[j] = wg + (int64_t)(col < c1 ? col : c1 - 1) * p.r + 8 * (q & 1);
      }
    }
    for (int s = 0; s < steps; ++s) {
      if constexpr (WT) {
        if (s % (kWtRanks / 16) == 0) {
          // the next ranks' rows of 64 columns into the wave's share: 8 lanes a row
          asm volatile("" ::: "memory");
          const int ranks = p.r - 16 * s < kWtRanks ? p.r - 16 * s : kWtRanks;
          for (int row = lane >> 3; row < (ranks + 15) / 16 * 16; row += 8) {
            const int col = n0 + (lane & 7) * 8;
            v4i v = v4i{0, 0, 0, 0};
            if (row < ranks && col < c1) v = load8(wg + (int64_t)(16 * s + row) * p.n + col);
            *reinterpret_cast<v4i*>(wt + row * 144 + (lane & 7) * 16) = v;
          }
          asm volatile("" ::: "memory");
        }
      }
      v4i wf[4], vf[MF];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (WT) {
          const uint8_t* at = wt + (s % (kWtRanks / 16) * 16 + 8 * (q & 1) + (x >> 2)) * 144 +
                              (32 * (j >> 1) + 8 * (x & 3) + 4 * (j & 1)) * 2;
          wf[j] = join(read_transposed(at), read_transposed(at + 4 * 144));
        } else {
          wf[j] = v4i{0, 0, 0, 0};
          if (16 * s + 8 * (q & 1) < p.r) wf[j] = load8(wp[j] + 16 * s);
        }
      }
#pragma unroll
      for (int i = 0; i < MF; ++i) vf[i] = *reinterpret_cast<const v4i*>(vt + (16 * i + x) * pitch + s * 64 + q * 16);
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = product16<F16>(wf[j], vf[i], acc[i][j]);
    }
#pragma unroll
    for (int jp = 0; jp < 2; ++jp)
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int col = n0 + 32 * jp + 8 * q;
        if (tok[i] < 0 || col >= c1) continue;
        const v4f a = acc[i][2 * jp], b = acc[i][2 * jp + 1];
        const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        v4i o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t u = (uint32_t)bs[jp][i][e];
          o[e] = (int)pack_half2<F16>(__builtin_fmaf(f[2 * e], back[i], half_lo<F16>(u)),
                                      __builtin_fmaf(f[2 * e + 1], back[i], half_hi<F16>(u)));
        }
        *reinterpret_cast<v4i*>(p.out + tok[i] * p.n + col) = o;
      }
  }
}

template <bool F16, int MF>
__global__ __launch_bounds__(kThreads) void lora_expand(ExpandArgs p) {
  if (blockIdx.x < p.tiles) expand_tile<F16, false, MF>(p, blockIdx.x);
  else expand_rest(p, (int)(blockIdx.x - p.tiles));
}

// ------------------------------------------------------------------ outer
// One chunk of an adapter's places: part[chunk] = sum over them of u[place, i]
// z[token, j], 16 RF ranks i and 128 columns j a workgroup, a wave 32 columns.  64
// places at a time: z's rows and u, cut into three BF16 parts that hold all its
// 24 bits, lie in LDS and are read transposed; FP16's z is cut into two BF16
// parts when it is read, and the products of the least parts (2^-24 of the
// value) left out.
struct OuterArgs {
  LoraPlan pl;
  const float* u;          // [slices, max_rows, r]
  const uint16_t* z;       // [m, k]
  float* part;             // [chunks, r, k]; UT: [chunks, k, r]
  int k, r, slices;
  int places;              // of a chunk
  unsigned tiles;          // workgroups
};
constexpr int kOuterCols = 128, kOuterRows = 64;

template <int RF>
constexpr int outer_smem() { return kOuterRows * (kOuterCols * 2 + 16) + 3 * kOuterRows * (RF * 32 + 16); }

template <bool F16, bool UT, int RF>
__device__ __forceinline__ void outer_tile(const OuterArgs& p, int id) {
  constexpr int ZP = kOuterCols * 2 + 16, UP = RF * 32 + 16;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), x = lane & 15, q = lane >> 4;
  const int kt = (p.k + kOuterCols - 1) / kOuterCols, rt = (p.r + 16 * RF - 1) / (16 * RF);
  const int j0 = id % kt * kOuterCols;
  id /= kt;
  const int i0 = id % rt * 16 * RF;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, p.places, id / rt);
  if (t.g < 0) return;
  const int end = t.row0 + p.places < t.row_end ? t.row0 + p.places : t.row_end;
  uint8_t* zt = smem;
  uint8_t* ut = smem + kOuterRows * ZP;
  v4f acc[RF][2];
#pragma unroll
  for (int i = 0; i < RF; ++i) acc[i][0] = acc[i][1] = v4f{0, 0, 0, 0};
  // a thread's pieces: 16 lanes a row of z (4 pieces), RF * 4 lanes a row of u (RF pieces of four values)
  v4i zr[4];
  v4f ur[RF];
  auto fetch = [&](int place0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int place = place0 + (tid >> 4) + 16 * e, col = j0 + (tid & 15) * 8;
      const int64_t tok = place < end ? token_at(p.pl, place) : -1;
      zr[e] = v4i{0, 0, 0, 0};
      if (tok >= 0 && col < p.k) zr[e] = load8(p.z + tok * p.k + col);
    }
#pragma unroll
    for (int e = 0; e < RF; ++e) {
      const int c = tid + 256 * e, place = place0 + c / (4 * RF), rank = i0 + c % (4 * RF) * 4;
      ur[e] = v4f{0, 0, 0, 0};
      if (place < end && rank < p.r && token_at(p.pl, place) >= 0) {
        const float* src = p.u + (int64_t)place * p.r + rank;
        ur[e] = *reinterpret_cast<const v4f*>(src);
        for (int s = 1; s < p.slices; ++s) ur[e] += *reinterpret_cast<const v4f*>(src + (int64_t)s * p.pl.max_rows * p.r);
      }
    }
  };
  fetch(t.row0);
  for (int place0 = t.row0; place0 < end; place0 += kOuterRows) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<v4i*>(zt + ((tid >> 4) + 16 * e) * ZP + (tid & 15) * 16) = zr[e];
#pragma unroll
    for (int e = 0; e < RF; ++e) {
      const int c = tid + 256 * e;
      uint8_t* d = ut + c / (4 * RF) * UP + c % (4 * RF) * 8;
      float v[4] = {ur[e][0], ur[e][1], ur[e][2], ur[e][3]};
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = __float_as_uint(v[i]) >> 16;
          if (v[i] != v[i]) h[i] |= 0x7fc0u;
          v[i] = bf16_rest(v[i], bf16_cut(v[i]));
        }
        *reinterpret_cast<uint2*>(d + part * kOuterRows * UP) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      }
    }
    __syncthreads();
    if (place0 + kOuterRows < end) fetch(place0 + kOuterRows);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 32 * h + 8 * q + (x >> 2);
      v4i zf[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* at = zt + row * ZP + (32 * w + 16 * j + 4 * (x & 3)) * 2;
        zf[j][0] = join(read_transposed(at), read_transposed(at + 4 * ZP));
        if constexpr (F16) {
          const v8h v = __builtin_bit_cast(v8h, zf[j][0]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = (float)v[2 * e], b = (float)v[2 * e + 1], ca = bf16_cut(a), cb = bf16_cut(b);
            uint32_t hi = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
            if (a != a) hi |= 0x7fc0u;
            if (b != b) hi |= 0x7fc00000u;
            zf[j][0][e] = (int)hi;
            zf[j][1][e] = (int)pack_half2<false>(bf16_rest(a, ca), bf16_rest(b, cb));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RF; ++i) {
        v4i uf[3];
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint8_t* at = ut + (part * kOuterRows + row) * UP + (16 * i + 4 * (x & 3)) * 2;
          uf[part] = join(read_transposed(at), read_transposed(at + 4 * UP));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          auto mul = [&](v4i u, v4i z) {
            acc[i][j] = UT ? product16<false>(u, z, acc[i][j]) : product16<false>(z, u, acc[i][j]);
          };
          if constexpr (F16) {
            mul(uf[1], zf[j][1]);
            mul(uf[0], zf[j][1]);
          }
          mul(uf[2], zf[j][0]);
          mul(uf[1], zf[j][0]);
          mul(uf[0], zf[j][0]);
        }
      }
    }
  }
  // four neighbours of a lane: columns (rank x) or, UT, ranks (column x)
  float* out = p.part + (int64_t)t.index * p.r * p.k;
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int rank = i0 + 16 * i + (UT ? 4 * q : x), col = j0 + 32 * w + 16 * j + (UT ? x : 4 * q);
      if (rank < p.r && col < p.k)
        *reinterpret_cast<v4f*>(out + (UT ? (int64_t)col * p.r + rank : (int64_t)rank * p.k + col)) = acc[i][j];
    }
}

// dx, dA's and dB's chunks in one launch: the longest first.
struct BackArgs {
  ExpandArgs dx;           // tiles and rest 0: no dx
  OuterArgs da, db;
};
template <bool F16, int MF, int RF>
__global__ __launch_bounds__(kThreads) void lora_back(BackArgs p) {
  unsigned id = blockIdx.x;
  if (id < p.da.tiles) return outer_tile<F16, false, RF>(p.da, (int)id);
  id -= p.da.tiles;
  if (id < p.db.tiles) return outer_tile<F16, true, RF>(p.db, (int)id);
  id -= p.db.tiles;
  if (id < p.dx.tiles) return expand_tile<F16, true, MF>(p.dx, (int)id);
  expand_rest(p.dx, (int)(id - p.dx.tiles));
}

// da, db: scale times the sum of an adapter's chunks, in order.
struct SumArgs {
  LoraPlan pl;
  const float *pa, *pb;
  float *da, *db;
  int64_t na, nb;          // values of an adapter
  int places;
  unsigned blocks;         // of an adapter
  bool accumulate;
};
__global__ __launch_bounds__(kThreads) void lora_sum(SumArgs p) {
  const int g = (int)(blockIdx.x / p.blocks);
  const int64_t at = ((int64_t)(blockIdx.x % p.blocks) * kThreads + threadIdx.x) * 4;
  const GroupTile t = group_tile<true>(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, p.places, g);
  if (at >= p.na + p.nb) return;
  const bool b = at >= p.na;
  const int64_t n = b ? p.nb : p.na, i = b ? at - p.na : at;
  const int chunks = (t.row_end - t.row0 + p.places - 1) / p.places;
  v4f* out = reinterpret_cast<v4f*>((b ? p.db : p.da) + g * n + i);
  if (p.accumulate && chunks == 0) return;
  const float* src = (b ? p.pb : p.pa) + t.first * n + i;
  v4f s = {0, 0, 0, 0};
  for (int c = 0; c < chunks; ++c) s += *reinterpret_cast<const v4f*>(src + c * n);
  const float f = p.pl.scale != nullptr ? p.pl.scale[g] : 1.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] *= f;
  if (p.accumulate) s += *out;
  *out = s;
}

// ------------------------------------------------------------------ plans
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
// At most this many tiles of bm places.
int64_t tile_bound(int64_t max_rows, int64_t adapters, int64_t bm) {
  return max_rows / bm + (max_rows < adapters ? max_rows : adapters);
}
constexpr int64_t kFill = 512;           // workgroups that fill the chip

int shrink_mf(int64_t max_rows, int64_t adapters) { return max_rows > 16 * adapters ? 2 : 1; }
int shrink_rf(int64_t r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }
int shrink_slices(int64_t max_rows, int64_t adapters, int64_t k, int64_t r) {
  const int64_t wgs = tile_bound(max_rows, adapters, 16 * shrink_mf(max_rows, adapters)) * up(r, 16 * shrink_rf(r));
  const int64_t most = up(k, 512);       // a block of 64 for each wave
  int64_t s = wgs > 0 ? kFill / wgs : 1;
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}
int expand_mf(int64_t max_rows, int64_t adapters, int64_t r) {
  return r > 256 || max_rows <= 16 * adapters ? 1 : r > 128 || max_rows <= 64 * adapters ? 2 : 4;
}
// Columns of a workgroup: 256, more where that leaves enough workgroups.
int expand_chunk(int64_t tiles, int64_t n) {
  int64_t c = 256;
  while (c < 4096 && c < n && tiles * up(n, 2 * c) >= 2 * kFill) c *= 2;
  return (int)c;
}
int outer_rf(int64_t r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }
// Places of a chunk of dA and dB: about 2 kFill workgroups.
int outer_places(int64_t max_rows, int64_t n, int64_t k, int64_t r) {
  const int64_t across = (up(n, kOuterCols) + up(k, kOuterCols)) * up(r, 16 * outer_rf(r));
  int64_t p = up(up(max_rows * across, 2 * kFill), 64) * 64;
  return (int)(p < 128 ? 128 : p > 8192 ? 8192 : p);
}

// More than 64 KB of dynamic LDS, allowed once per device (twice is harmless).
template <class K>
hipError_t allow_smem(K kernel, int bytes, std::atomic<bool> (&set)[64]) {
  if (bytes <= 65536) return hipSuccess;
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  if (cached && set[dev].load(std::memory_order_acquire)) return hipSuccess;
  e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && cached) set[dev].store(true, std::memory_order_release);
  return e;
}

template <bool F16, bool WT, int MF, int RF>
hipError_t shrink_one(hipStream_t s, const ShrinkArgs& p) {
  constexpr int kSum = kShrinkWaves * MF * RF * 1024, kW = WT ? kShrinkWaves * 64 * (RF * 32 + 16) : 0;
  constexpr int bytes = kSum > kW ? kSum : kW;
  const int64_t wgs = tile_bound(p.pl.max_rows, p.pl.adapters, 16 * MF) * up(p.r, 16 * RF) * p.slices;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_smem(lora_shrink<F16, WT, MF, RF>, bytes, set);
  if (e != hipSuccess || wgs == 0) return e;
  hipLaunchKernelGGL((lora_shrink<F16, WT, MF, RF>), dim3((unsigned)wgs), dim3(kShrinkWaves * 64), bytes, s, p);
  return hipGetLastError();
}
template <bool F16, bool WT>
hipError_t shrink(hipStream_t s, const ShrinkArgs& p) {
  const int mf = shrink_mf(p.pl.max_rows, p.pl.adapters), rf = shrink_rf(p.r);
  if (mf == 1) return rf == 1 ? shrink_one<F16, WT, 1, 1>(s, p) : rf == 2 ? shrink_one<F16, WT, 1, 2>(s, p) : shrink_one<F16, WT, 1, 4>(s, p);
  return rf == 1 ? shrink_one<F16, WT, 2, 1>(s, p) : rf == 2 ? shrink_one<F16, WT, 2, 2>(s, p) : shrink_one<F16, WT, 2, 4>(s, p);
}

ExpandArgs expand_args(const LoraPlan& pl, const float* v, const uint16_t* w, const uint16_t* base, uint16_t* out,
                       float* v_out, int64_t n, int64_t r, int slices) {
  ExpandArgs p{pl, v, w, base, out, v_out, (int)n, (int)r, slices, 0, 0, 0, 0};
  const int64_t tiles = tile_bound(pl.max_rows, pl.adapters, 16 * expand_mf(pl.max_rows, pl.adapters, r));
  p.chunk = expand_chunk(tiles, n);
  p.chunks = (int)up(n, p.chunk);
  p.tiles = (unsigned)(tiles * p.chunks);
  p.rest = base != out ? (unsigned)(up(pl.m, kRestRows) * p.chunks) : 0;
  return p;
}

template <bool F16, int MF>
hipError_t expand_one(hipStream_t s, const ExpandArgs& p) {
  const int bytes = expand_smem<false, MF>(p.r);
  if (p.tiles + p.rest == 0) return hipSuccess;
  hipLaunchKernelGGL((lora_expand<F16, MF>), dim3(p.tiles + p.rest), dim3(kThreads), bytes, s, p);
  return hipGetLastError();
}
template <bool F16>
hipError_t forward(hipStream_t s, const LoraArgs& p) {
  const LoraPlan& pl = p.plan;
  const int slices = shrink_slices(pl.max_rows, pl.adapters, p.k, p.r);
  float* v = slices == 1 && p.v != nullptr ? p.v : static_cast<float*>(p.workspace);
  const hipError_t e = shrink<F16, false>(s, ShrinkArgs{pl, p.x, p.a, v, (int)p.k, (int)p.r, slices});
  if (e != hipSuccess) return e;
  const ExpandArgs x = expand_args(pl, v, p.b, p.base, p.out, v != p.v ? p.v : nullptr, p.n, p.r, slices);
  switch (expand_mf(pl.max_rows, pl.adapters, p.r)) {
    case 1: return expand_one<F16, 1>(s, x);
    case 2: return expand_one<F16, 2>(s, x);
    default: return expand_one<F16, 4>(s, x);
  }
}

template <bool F16, int MF, int RF>
hipError_t back_one(hipStream_t s, const BackArgs& p) {
  const int a = expand_smem<true, MF>(p.dx.r), b = outer_smem<RF>(), bytes = a > b ? a : b;
  const unsigned wgs = p.da.tiles + p.db.tiles + p.dx.tiles + p.dx.rest;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_smem(lora_back<F16, MF, RF>, bytes > 65536 ? 163840 : bytes, set);
  if (e != hipSuccess || wgs == 0) return e;
  hipLaunchKernelGGL((lora_back<F16, MF, RF>), dim3(wgs), dim3(kThreads), bytes, s, p);
  return hipGetLastError();
}
template <bool F16, int MF>
hipError_t back(hipStream_t s, const BackArgs& p) {
  const int rf = outer_rf(p.dx.r);
  return rf == 1 ? back_one<F16, MF, 1>(s, p) : rf == 2 ? back_one<F16, MF, 2>(s, p) : back_one<F16, MF, 4>(s, p);
}

struct BackSpace {
  uint64_t u, da, db;      // bytes
};
BackSpace back_space(int64_t max_rows, int64_t n, int64_t k, int64_t r, int64_t adapters) {
  const int64_t chunks = tile_bound(max_rows, adapters, outer_places(max_rows, n, k, r));
  return {(uint64_t)shrink_slices(max_rows, adapters, n, r) * max_rows * r * 4, (uint64_t)chunks * r * k * 4,
          (uint64_t)chunks * r * n * 4};
}

template <bool F16>
hipError_t backward(hipStream_t s, const LoraArgs& p) {
  const LoraPlan& pl = p.plan;
  const BackSpace sp = back_space(pl.max_rows, p.n, p.k, p.r, pl.adapters);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  float *u = reinterpret_cast<float*>(ws), *pa = reinterpret_cast<float*>(ws + sp.u), *pb = reinterpret_cast<float*>(ws + sp.u + sp.da);
  const int slices = shrink_slices(pl.max_rows, pl.adapters, p.n, p.r);
  hipError_t e = shrink<F16, true>(s, ShrinkArgs{pl, p.dy, p.b, u, (int)p.n, (int)p.r, slices});
  if (e != hipSuccess) return e;
  BackArgs x{};
  x.dx = expand_args(pl, u, p.a, p.base, p.out, nullptr, p.k, p.r, slices);
  if (p.out == nullptr) x.dx.tiles = x.dx.rest = 0;
  const int places = outer_places(pl.max_rows, p.n, p.k, p.r);
  const int64_t each = tile_bound(pl.max_rows, pl.adapters, places) * up(p.r, 16 * outer_rf(p.r));
  x.da = OuterArgs{pl, u, p.x, pa, (int)p.k, (int)p.r, slices, places, (unsigned)(each * up(p.k, kOuterCols))};
  x.db = OuterArgs{pl, p.v, p.dy, pb, (int)p.n, (int)p.r, 1, places, (unsigned)(each * up(p.n, kOuterCols))};
  switch (expand_mf(pl.max_rows, pl.adapters, p.r)) {
    case 1: e = back<F16, 1>(s, x); break;
    case 2: e = back<F16, 2>(s, x); break;
    default: e = back<F16, 4>(s, x); break;
  }
  if (e != hipSuccess) return e;
  SumArgs m{pl, pa, pb, p.da, p.db, p.r * p.k, p.r * p.n, places, (unsigned)up(p.r * (p.k + p.n), 4 * kThreads), p.accumulate};
  hipLaunchKernelGGL(lora_sum, dim3(m.blocks * (unsigned)pl.adapters), dim3(kThreads), 0, s, m);
  return hipGetLastError();
}

}  // namespace

// The most work items of a launch of either direction.
int64_t lora_work_items(int64_t max_rows, int64_t m, int64_t n, int64_t k, int64_t r, int64_t adapters) {
  auto more = [](int64_t& most, int64_t wgs, int64_t threads) {
    const int64_t v = wgs < ((int64_t)1 << 40) ? wgs * threads : (int64_t)1 << 50;
    most = v > most ? v : most;
  };
  int64_t most = 0;
  const int64_t tiles = tile_bound(max_rows, adapters, 16 * expand_mf(max_rows, adapters, r));
  const int64_t places = outer_places(max_rows, n, k, r), chunks = tile_bound(max_rows, adapters, places);
  for (const int64_t inner : {n, k})
    more(most, tile_bound(max_rows, adapters, 16 * shrink_mf(max_rows, adapters)) * up(r, 16 * shrink_rf(r)) *
                   shrink_slices(max_rows, adapters, inner, r), kShrinkWaves * 64);
  int64_t back = chunks * up(r, 16 * outer_rf(r)) * (up(n, kOuterCols) + up(k, kOuterCols));
  for (const int64_t outer : {n, k}) {
    const int64_t wgs = (tiles + up(m, kRestRows)) * up(outer, expand_chunk(tiles, outer));
    more(most, wgs, kThreads);
    if (outer == k) back += wgs;
  }
  more(most, back, kThreads);
  more(most, up(r * (k + n), 4 * kThreads) * adapters, kThreads);
  return most;
}

uint64_t lora_workspace_bytes(int64_t max_rows, int64_t, int64_t k, int64_t r, int32_t adapters) {
  return (uint64_t)shrink_slices(max_rows, adapters, k, r) * max_rows * r * 4;
}
uint64_t lora_backward_workspace_bytes(int64_t max_rows, int64_t n, int64_t k, int64_t r, int32_t adapters) {
  const BackSpace sp = back_space(max_rows, n, k, r, adapters);
  return sp.u + sp.da + sp.db;
}

hipError_t launch_lora(hipStream_t s, const LoraArgs& p) { return p.f16 ? forward<true>(s, p) : forward<false>(s, p); }
hipError_t launch_lora_backward(hipStream_t s, const LoraArgs& p) {
  return p.f16 ? backward<true>(s, p) : backward<false>(s, p);
}

}  // namespace hq
