// Block-128 FP8 quantisation of BF16 / FP16 tensors [batch, m, k]: 1 x 128
// blocks along the rows or 128 x 128 blocks, with the codes in x's layout or
// transposed, and the SwiGLU of a gate|up row quantised in 1 x 128 blocks.
//
// Every form reads its input once and writes codes and scales once: 3 bytes
// an element (5 for SwiGLU outputs).  A large copy reaches 5.1 TB/s.  Memory
// bounds the row form, also with partial blocks, SwiGLU, and tiles whose rows are
// whole lines of x and q: [65536, 4096] rows 132 us, 6.2 TB/s; SwiGLU of [65536, 2 x
// 1536] 90 us, 5.6; 32 x [4096, 1536] in 128 x 128 blocks 109 us, transposed 103.
// Tiles fall behind it otherwise: a tile row's 256 bytes of x straddle lines
// where k % 64 != 0, and a row's 128 bytes of codes are parts of lines where q's
// rows are not a multiple of 128 bytes ([16416, 4128] against [16384, 4096], us: 128 x
// 128 50.8, 39.7; transposed 48.3, 41.4; 1 x 128 transposed 52.2, 42.0); 1 x 128
// transposed also writes its scales one by one into as many lines ([65536, 4096]
// 181 us, 4.5 TB/s).  Up to about 20 MB launch and latency are half of the time
// ([4096, 1536] 6 to 7 us for 3.7).
#include "block_fmt.hpp"
#include "block_internal.hpp"

namespace hq {
namespace {

constexpr int kThreads = kQuantThreads;

// Row form, and SwiGLU (x [rows, 2k] = [gate | up], y = up * silu(gate)).
// Eight lanes take a 128-block, 16 values each: two 16-byte loads, one 16-byte
// store of codes, and an amax over the lane octet in three DPP steps.
// Octets are numbered along the whole tensor, so any k (a multiple of 32)
// keeps every lane busy but those past a row's last partial block.
template <bool F16, bool SWIGLU, bool NT>
__global__ __launch_bounds__(kThreads) void block_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t k,
                                                              int32_t nkb, const int32_t* __restrict__ last_end,
                                                              uint8_t* __restrict__ q, float* __restrict__ sf) {
  const uint32_t o = blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3);      // below 2^29
  const int l = threadIdx.x & 7;
  const int64_t row = o / (uint32_t)nkb;
  const int kb = (int)(o - (uint32_t)row * (uint32_t)nkb);
  if (last_end != nullptr) {
    const int64_t e = *last_end;
    rows = e < 0 ? 0 : (e < rows ? e : rows);
  }
  const int64_t c = (int64_t)kb * 128 + l * 16;
  const bool in = row < rows && c < k;
  float f[16];
  uint32_t mx = 0;
  if (in) {
    const uint4* p = reinterpret_cast<const uint4*>(x + row * (SWIGLU ? 2 * k : k) + c);
    const uint4 v0 = load_nt(p), v1 = load_nt(p + 1);
    unpack16<F16>(v0, v1, f);
    if constexpr (SWIGLU) {
      const uint4* pu = reinterpret_cast<const uint4*>(x + row * 2 * k + k + c);
      float u[16];
      unpack16<F16>(load_nt(pu), load_nt(pu + 1), u);
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = silu_mul(f[i], u[i]);
      mx = abs_max(f);
    } else {
      mx = abs_max<F16>(v0, v1);
    }
  }
  const float s = block_scale(octet_max_u32(mx));
  if (!in) return;
  uint32_t w[4];
  block_codes(f, s, w);
  store16<NT>(q + row * k + c, u32x4{w[0], w[1], w[2], w[3]});
  if (l == 0) sf[row * nkb + kb] = s;
}

// Tile forms: one workgroup takes a 128 x 128 tile of x (rows m0.., columns
// k0.. of one batch item).  Pass p of four gives lane octet (thread / 8) the
// tile row 32 p + thread / 8, 16 values a lane.
//   TRANS = false: one scale per tile (128 x 128 blocks), codes in x's layout.
//   A lane's two loads share a cache line, which non-temporal ones did not keep
//   between them (32 x [4096, 1536] 115.4 -> 109.5 us); the row form and the
//   transposes measured 1 to 5 % slower with plain loads above 100 MB.
//   TRANS = true: the codes go through LDS and leave as rows of q [k, m]; the
//   scale is per tile (TWO_D) or per column of x (1 x 128 blocks of q's rows).
template <bool F16, bool TWO_D, bool TRANS, bool NT>
__global__ __launch_bounds__(kThreads) void block_tile_kernel(const uint16_t* __restrict__ x, int64_t m, int64_t k,
                                                              int32_t tiles_m, int32_t tiles_k,
                                                              uint8_t* __restrict__ q, float* __restrict__ sf) {
  static_assert(TWO_D || TRANS, "the row form has a kernel of its own");
  __shared__ uint32_t red[TWO_D ? kThreads / 64 : 4 * 128];
  __shared__ __attribute__((aligned(16))) uint32_t lt[TRANS ? 128 * 36 : 1];   // codes: column c's 128 bytes at 144 c
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t t = blockIdx.x;
  const int64_t bt = t / ((int64_t)tiles_m * tiles_k);
  const int rem = (int)(t - bt * tiles_m * tiles_k);
  const int tm = rem / tiles_k, tk = rem - tm * tiles_k;
  const int64_t m0 = (int64_t)tm * 128, k0 = (int64_t)tk * 128;
  const uint16_t* xb = x + bt * m * k;
  uint8_t* qb = q + bt * m * k;

  if constexpr (!TRANS) {
    const int l = tid & 7, r8 = tid >> 3;
    const int64_t c = k0 + l * 16;
    uint4 v[4][2];
    uint32_t mx = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int64_t r = m0 + 32 * p + r8;
      v[p][0] = v[p][1] = make_uint4(0, 0, 0, 0);
      if (r < m && c < k) {
        const uint4* s = reinterpret_cast<const uint4*>(xb + r * k + c);
        v[p][0] = s[0];
        v[p][1] = s[1];
      }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t a = abs_max<F16>(v[p][0], v[p][1]);
      mx = a > mx ? a : mx;
    }
    mx = wave_max_u32(mx);
    if (lane == 0) red[w] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) mx = red[i] > mx ? red[i] : mx;
    const float s = block_scale(mx);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int64_t r = m0 + 32 * p + r8;
      if (r < m && c < k) {
        float f[16];
        unpack16<F16>(v[p][0], v[p][1], f);
        uint32_t o[4];
        block_codes(f, s, o);
        store16<NT>(qb + r * k + c, u32x4{o[0], o[1], o[2], o[3]});
      }
    }
    if (tid == 0) sf[(bt * tiles_m + tm) * tiles_k + tk] = s;
    return;
  } else {
    // Lane c2 of every wave owns columns 2 c2 and 2 c2 + 1; wave w the tile
    // rows 32 w .. 32 w + 31, one dword (a column pair) a row.
    const int64_t c = k0 + 2 * lane;
    uint32_t v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int64_t r = m0 + 32 * w + i;
      v[i] = r < m && c < k ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(xb + r * k + c)) : 0u;
    }
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m2 = abs_max2(m2, v[i]);
    uint32_t mlo = __float_as_uint(half_lo<F16>(m2)), mhi = __float_as_uint(half_hi<F16>(m2));
    float slo, shi;
    if constexpr (TWO_D) {
      uint32_t mx = wave_max_u32(mlo > mhi ? mlo : mhi);
      if (lane == 0) red[w] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kThreads / 64; ++i) mx = red[i] > mx ? red[i] : mx;
      slo = shi = block_scale(mx);
      if (tid == 0) sf[(bt * tiles_k + tk) * tiles_m + tm] = slo;
    } else {
      red[w * 128 + 2 * lane] = mlo;
      red[w * 128 + 2 * lane + 1] = mhi;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = red[i * 128 + 2 * lane], b = red[i * 128 + 2 * lane + 1];
        mlo = a > mlo ? a : mlo;
        mhi = b > mhi ? b : mhi;
      }
      slo = block_scale(mlo);
      shi = block_scale(mhi);
      if (w == 0 && c < k) {
        sf[(bt * k + c) * tiles_m + tm] = slo;
        sf[(bt * k + c + 1) * tiles_m + tm] = shi;
      }
    }
    float f[32];
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = half_lo<F16>(v[i]);
    block_codes(f, slo, o);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(lt + (2 * lane) * 36 + 8 * w + 4 * i) =
          make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = half_hi<F16>(v[i]);
    block_codes(f, shi, o);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(lt + (2 * lane + 1) * 36 + 8 * w + 4 * i) =
          make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    __syncthreads();
    // out: octet (thread / 8) writes 128 bytes of q's row k0 + 32 p + thread / 8
    const int l = tid & 7, r8 = tid >> 3;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int cc = 32 * p + r8;
      if (k0 + cc < k && m0 + 16 * l < m)
        store16<NT>(qb + (k0 + cc) * m + m0 + 16 * l, *reinterpret_cast<const u32x4*>(lt + cc * 36 + 4 * l));
    }
  }
}

template <bool SWIGLU>
hipError_t launch_rows(hipStream_t s, const uint16_t* x, int64_t rows, int64_t k, const int32_t* last_end, uint8_t* q,
                       float* sf, bool fp16) {
  const int64_t nkb = (k + 127) / 128, blocks = quant_row_groups(rows, k);
  const bool nt = rows * k > kStreamBytes;
#define HQ_ROWS(F, N)                                                                                                \
  hipLaunchKernelGGL((block_rows_kernel<F, SWIGLU, N>), dim3((unsigned)blocks), dim3(kThreads), 0, s, x, rows, k,   \
                     (int32_t)nkb, last_end, q, sf)
  if (fp16 && nt) HQ_ROWS(true, true);
  else if (fp16) HQ_ROWS(true, false);
  else if (nt) HQ_ROWS(false, true);
  else HQ_ROWS(false, false);
#undef HQ_ROWS
  return hipGetLastError();
}

template <bool TWO_D, bool TRANS>
hipError_t launch_tiles(hipStream_t s, const uint16_t* x, int64_t batch, int64_t m, int64_t k, uint8_t* q, float* sf,
                        bool fp16) {
  const int64_t tk = (k + 127) / 128, tm = (m + 127) / 128;
  const bool nt = batch * m * k > kStreamBytes;
#define HQ_TILE(F, N)                                                                                          \
  hipLaunchKernelGGL((block_tile_kernel<F, TWO_D, TRANS, N>), dim3((unsigned)quant_tile_groups(batch, m, k)),          \
                     dim3(kThreads), 0, s, x, m, k, (int32_t)tm, (int32_t)tk, q, sf)
  if (fp16 && nt) HQ_TILE(true, true);
  else if (fp16) HQ_TILE(true, false);
  else if (nt) HQ_TILE(false, true);
  else HQ_TILE(false, false);
#undef HQ_TILE
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_quant(hipStream_t s, const uint16_t* x, int64_t batch, int64_t m, int64_t k, uint8_t* q,
                              float* sf, bool two_d, bool transpose, bool fp16) {
  if (two_d && transpose) return launch_tiles<true, true>(s, x, batch, m, k, q, sf, fp16);
  if (two_d) return launch_tiles<true, false>(s, x, batch, m, k, q, sf, fp16);
  if (transpose) return launch_tiles<false, true>(s, x, batch, m, k, q, sf, fp16);
  return launch_rows<false>(s, x, batch * m, k, nullptr, q, sf, fp16);
}

hipError_t launch_swiglu_block_quant(hipStream_t s, const uint16_t* x, int64_t rows, int64_t h,
                                     const int32_t* last_end, uint8_t* q, float* sf, bool fp16) {
  return launch_rows<true>(s, x, rows, h, last_end, q, sf, fp16);
}

}  // namespace hq
