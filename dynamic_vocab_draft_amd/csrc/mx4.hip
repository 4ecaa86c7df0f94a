// 4-bit rows: microscaled floating point.  Quantisation, rows read back, the
// product, and the restricted LM head over 4-bit rows.
//
// 32 consecutive elements share a power of two.  With a = max |x_i| of a block
//     e = floor(log2 a) - 2  (at least -127; -127 for a block of zeros),
//     q_i = x_i / 2^e to E2M1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives),
//           nearest, halfway cases to the even code, 6 beyond 6,
// and the scale is kept as the byte e + 127, 255 for a block with a NaN or an
// infinity, whose products are NaN.  The product
//     out[m, n] = sum_b 2^(ex[m, b] + ew[n, b]) sum_{i in b} xq[m, i] wq[n, i]
// is one scaled matrix instruction for every 128 elements.  Products of two
// codes are quarters of integers up to 144, so a float32 sum is exact, however it
// was split, while 144 d 2^s <= 2^24, where the terms' scales lie within 2^s of one
// another: s = 4 at d = 4096.  Rows of random signs, whose sums grow as sqrt(d), stay
// exact further, to some 2^10.
#include <type_traits>

#include "common.hpp"
#include "head_top.hpp"
#include "lds_loads.hpp"
#include "rows.hpp"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kChunk = 256;                        // elements: 128 bytes of codes, 8 scales
constexpr int kChunkBytes = kChunk / 2, kChunkScales = kChunk / 32;
__host__ __device__ constexpr int chunks_of(int d) { return (d + kChunk - 1) / kChunk; }
__host__ __device__ constexpr int pitch_of(int d) { return chunks_of(d) * kChunkBytes; }

// ---------------------------------------------------------------------------
// Quantisation: one pass, bound by its bytes (128256 x 4096 bf16 228 to 245 us,
// 5.4 to 5.8 TB/s read and written).  A lane takes eight elements, four lanes a block, so a row's
// 256-element chunk is half a wave's.  Of float32 a lane takes four in each half
// of the chunk, so that a load of all lanes is one run of the row.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
// Chunks of a half wave: many where there are enough to fill the chip, else one,
// whose blocks are more and end sooner.
constexpr int kManyUnits = 8, kManyChunks = 1 << 17;

// c / d for c < 2^26 and d <= 64, from 2^32 / d rounded up: the quotient is over
// by less than c / 2^32 < 1 / d.  0 stands for 2^32.
__host__ __device__ __forceinline__ uint32_t reciprocal_of(uint32_t d) { return d == 1 ? 0u : 0xFFFFFFFFu / d + 1u; }
__device__ __forceinline__ uint32_t divided(uint32_t c, uint32_t rcp) { return rcp == 0 ? c : __umulhi(c, rcp); }

// The largest value of four lanes.
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);    // quad_perm 1 0 3 2
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);             // quad_perm 2 3 0 1
  return o > v ? o : v;
}

// The largest value of eight lanes.
__device__ __forceinline__ uint32_t oct_max_u32(uint32_t v) {
  v = quad_max_u32(v);
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true);   // row_half_mirror
  return o > v ? o : v;
}

// The scale byte from the float32 bits of the block's largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;                    // biased; 255 for infinities and NaN
  return e == 255 ? 255u : (e > 2 ? e - 2 : 0u);
}

// 2^(byte - 127) as a float, the smallest one a subnormal; not for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// Eight elements to eight codes, the first in the lowest bits.
template <int ET>
__device__ __forceinline__ uint32_t quant_eight(const Eight<ET>& x, uint32_t byte) {
  const float s = scale_value(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(0), x.get(1), s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(2), x.get(3), s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(4), x.get(5), s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(6), x.get(7), s, 3);
  return byte == 255 ? 0u : r;
}

// The largest magnitude of eight elements, as float32 bits, which order like it.
template <int ET>
__device__ __forceinline__ uint32_t top_bits(const Eight<ET>& x) {
  const uint32_t m = x.top(0);
  if (ET == NS_FP32) return m;
  const uint32_t lo = m & 0xFFFFu, hi = m >> 16, b = lo > hi ? lo : hi;
  return __float_as_uint(ET == NS_BF16 ? ns::bf16_lo(b) : ns::fp16_lo(b));
}

// A chunk of a row by half a wave, lane l of it: its codes and scales.
template <int ET>
__device__ __forceinline__ void put_chunk(const Eight<ET>& v, int l, uint8_t* to, uint8_t* scale) {
  if constexpr (ET == NS_FP32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t t = v.v[h][e] & 0x7FFFFFFFu;
        top = t > top ? t : top;
      }
      const uint32_t byte = scale_byte(oct_max_u32(top));
      const float f = scale_value(byte);
      uint32_t r = 0;
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v.get(4 * h), v.get(4 * h + 1), f, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v.get(4 * h + 2), v.get(4 * h + 3), f, 1);
      *(uint16_t*)(to + h * (kChunkBytes / 2) + l * 2) = byte == 255 ? (uint16_t)0 : (uint16_t)r;
      if ((l & 7) == 0) scale[h * (kChunkScales / 2) + (l >> 3)] = (uint8_t)byte;
    }
  } else {
    const uint32_t byte = scale_byte(quad_max_u32(top_bits<ET>(v)));
    *(uint32_t*)(to + l * 4) = quant_eight<ET>(v, byte);
    if ((l & 3) == 0) scale[l >> 2] = (uint8_t)byte;
  }
}

template <int ET, int UNITS>
__global__ __launch_bounds__(kRowThreads) void k_mx4_rows(const void* __restrict__ x, int64_t ld, int R, int d,
                                                          uint32_t rcp, uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ scale) {
  const int per_row = chunks_of(d), total = R * per_row;   // below 2^26
  const int l = threadIdx.x & 31, c0 = (int)blockIdx.x * (kRowThreads / 32 * UNITS) + (threadIdx.x >> 5);
  const int tail = d & ~(ET == NS_FP32 ? 3 : 7);
  Eight<ET> v[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = c0 + u * (kRowThreads / 32), cc = c < total ? c : total - 1;
    const int r = (int)divided((uint32_t)cc, rcp);
    const char* row = (const char*)x + (size_t)r * (size_t)ld * (ET == NS_FP32 ? 4 : 2);
    v[u].load(row, (cc - r * per_row) * kChunk + l * (ET == NS_FP32 ? 4 : 8), kChunk / 2, tail, Eight<ET>::rest_of(row, tail, d));
  }
  NS_ISSUE_FENCE();
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = c0 + u * (kRowThreads / 32);
    if (c >= total) continue;                      // whole half waves
    put_chunk<ET>(v[u], l, q + (size_t)c * kChunkBytes, scale + (size_t)c * kChunkScales);
  }
}

template <int ET>
void launch_rows(const void* x, int64_t ld, int R, int d, uint8_t* q, uint8_t* scale, hipStream_t stream) {
  const int total = R * chunks_of(d), groups = kRowThreads / 32;
  const uint32_t rcp = reciprocal_of((uint32_t)chunks_of(d));
  const auto blocks = [&](int units) { return dim3((unsigned)((total + groups * units - 1) / (groups * units))); };
  if (total >= kManyChunks) hipLaunchKernelGGL((k_mx4_rows<ET, kManyUnits>), blocks(kManyUnits), dim3(kRowThreads), 0, stream, x, ld, R, d, rcp, q, scale);
  else hipLaunchKernelGGL((k_mx4_rows<ET, 1>), blocks(1), dim3(kRowThreads), 0, stream, x, ld, R, d, rcp, q, scale);
}

int mx4_rows(const void* x, int64_t ld, int R, int d, int dtype, uint8_t* q, uint8_t* scale, hipStream_t stream) {
  if (dtype == NS_BF16) launch_rows<NS_BF16>(x, ld, R, d, q, scale, stream);
  else if (dtype == NS_FP16) launch_rows<NS_FP16>(x, ld, R, d, q, scale, stream);
  else launch_rows<NS_FP32>(x, ld, R, d, q, scale, stream);
  return ns_launch_status();
}

// ---------------------------------------------------------------------------
// Rows read back: out[j, :] = values of row ids[j].
// ---------------------------------------------------------------------------
// Eight codes to eight values.
__device__ __forceinline__ void values_of(uint32_t codes, uint32_t byte, float (&v)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float s = scale_value(byte), nan = __uint_as_float(0x7FC00000u);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 3);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y; v[4] = c.x; v[5] = c.y; v[6] = e.x; v[7] = e.y;
  if (byte == 255) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = nan;
  }
}

// A lane takes eight elements, of float32 four in each half of the chunk, so that
// a store of all lanes is one run of the row.  Nobody reads the outputs soon:
// stores past the caches (128256 x 4096 bf16 294 -> 217 us, 6.1 TB/s), but for float32
// rows that share lines (60000 x 1001, quantised and read back, 132 us past them, 106
// through them; 4095 bf16 elements 345 and 373).
template <int OT, int UNITS, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void k_mx4_gather(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                            int V, int d, uint32_t rcp, const int32_t* __restrict__ ids,
                                                            const int32_t* __restrict__ n_dev, int n_max,
                                                            void* __restrict__ out, int64_t ld) {
  constexpr bool F32 = OT == NS_FP32;
  const int per_row = chunks_of(d);
  int n = n_dev ? *n_dev : n_max;
  n = n < 0 ? 0 : (n > n_max ? n_max : n);
  const int total = n * per_row;                   // below 2^26
  const int l = threadIdx.x & 31, c0 = (int)blockIdx.x * (kRowThreads / 32 * UNITS) + (threadIdx.x >> 5);
  uint32_t codes[UNITS], byte[UNITS];              // of float32 two halves in each
  int row[UNITS], at[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = c0 + u * (kRowThreads / 32);
    row[u] = -1;
    if (c >= total) continue;
    const int j = (int)divided((uint32_t)c, rcp), id = ids ? ids[j] : j;
    at[u] = (c - j * per_row) * kChunk;
    if (id < 0 || id >= V) continue;
    const size_t from = (size_t)id * per_row + (c - j * per_row);
    const uint8_t *f = q + from * kChunkBytes, *b = scale + from * kChunkScales;
    if (F32) {
      codes[u] = (uint32_t)__builtin_nontemporal_load((const uint16_t*)(f + l * 2)) |
                 (uint32_t)__builtin_nontemporal_load((const uint16_t*)(f + kChunkBytes / 2 + l * 2)) << 16;
      byte[u] = (uint32_t)b[l >> 3] | (uint32_t)b[kChunkScales / 2 + (l >> 3)] << 8;
    } else {
      codes[u] = __builtin_nontemporal_load((const uint32_t*)(f + l * 4));
      byte[u] = b[l >> 2];
    }
    row[u] = j;
  }
  NS_ISSUE_FENCE();
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    if (row[u] < 0) continue;
    const size_t base = (size_t)row[u] * (size_t)ld;
    float v[8];
    if constexpr (F32) {
      float w[8];
      values_of(codes[u], byte[u] & 255, v);       // the lower half's four
      values_of(codes[u], byte[u] >> 8, w);        // and, behind four of no use, the upper's
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = at[u] + h * (kChunk / 2) + l * 4;
        const float* x = h == 0 ? v : w + 4;
        float* to = (float*)out + base + i;
        if (d - i >= 4) {
          const u32x4 y = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
          if (ONCE) __builtin_nontemporal_store(y, (u32x4_any*)to);
          else *(u32x4_any*)to = y;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < d - i) to[e] = x[e];
        }
      }
    } else {
      const int i = at[u] + l * 8;
      if (i >= d) continue;
      values_of(codes[u], byte[u], v);
      if (d - i >= 8) {
        __builtin_nontemporal_store(u32x4{narrow2<OT>(v[0], v[1]), narrow2<OT>(v[2], v[3]), narrow2<OT>(v[4], v[5]), narrow2<OT>(v[6], v[7])},
                                    (u32x4_any*)((uint16_t*)out + base + i));
      } else {
        store_eight<OT>(out, base + i, v, d - i);
      }
    }
  }
}

template <int OT>
void launch_gather(const uint8_t* q, const uint8_t* scale, int V, int d, const int32_t* ids, const int32_t* n_dev, int n_max, void* out,
                   int64_t ld, hipStream_t stream) {
  const int total = n_max * chunks_of(d), groups = kRowThreads / 32;
  const uint32_t rcp = reciprocal_of((uint32_t)chunks_of(d));
  const auto blocks = [&](int units) { return dim3((unsigned)((total + groups * units - 1) / (groups * units))); };
  const auto go = [&](auto units, auto once) {
    hipLaunchKernelGGL((k_mx4_gather<OT, decltype(units)::value, decltype(once)::value>), blocks(decltype(units)::value), dim3(kRowThreads), 0,
                       stream, q, scale, V, d, rcp, ids, n_dev, n_max, out, ld);
  };
  const bool once = OT != NS_FP32 || ((uint64_t)(uintptr_t)out | (uint64_t)ld * 4) % 128 == 0;
  if (total < kManyChunks) go(std::integral_constant<int, 1>(), std::true_type());
  else if (once) go(std::integral_constant<int, kManyUnits>(), std::true_type());
  else go(std::integral_constant<int, kManyUnits>(), std::integral_constant<bool, OT != NS_FP32>());
}

// ---------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------
struct Product {
  const uint8_t* x;         // [B][M][pitch]
  const uint8_t* xs;        // [B][M][pitch / 16]
  const uint8_t* w;         // [rows][pitch]
  const uint8_t* ws;        // [rows][pitch / 16]
  const int32_t* ids;       // [B][N] row of column j, or NULL: j
  const int32_t* n_dev;     // [B] live columns, or NULL: N
  int M, N, V, pitch;
  void* out;                // [B][M][N], elements of a token `sm` apart for m, `sn` for n
  int64_t sm, sn;
};

// 16 x 16 outputs over 128 elements.  Lane (i, g) holds 32 elements of row i of
// each operand, one block, and byte BYTE of sa and sb is that block's scale;
// which elements a place holds is free as long as both operands agree.
template <int BYTE>
__device__ __forceinline__ f32x4 product128(i32x4 a, i32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, BYTE, (int)sa, BYTE, (int)sb);
}

// Two scales as an operand, whose upper half is nobody's.  A pair, not an integer,
// so that no instruction clears that half (1.6 % of 4096 x 16384 x 16384).
__device__ __forceinline__ u16x2 two_scales(const char* p) {
  u16x2 r;
  r.x = *(const uint16_t*)p;
  return r;
}

// ---------------------------------------------------------------------------
// The product for few channel rows: bound by latency (4 x 2048 x 256 3.0 us, one
// trip to memory and the joining of the sums).  A block of eight waves owns 16
// channel rows and up to 64 token rows (blockIdx.z of them); each wave takes an
// eighth of the row's chunks, asks for BATCH of them at once and multiplies; the
// eight sums are joined in LDS.  Loads are whole lines, eight lanes a row, and pass
// through LDS to the lanes that multiply them, without a word to another wave (lanes
// that loaded what they multiply touched 64 lines a load: 64 x 4096 x 16384 29.1 ->
// 18.8 us, 8 x 8000 x 4096 7.2 -> 5.4; 64 x 200 x 256 3.2 -> 3.6).  Lane (i, g)
// multiplies blocks 2 g and 2 g + 1 of row i's chunk.
// ---------------------------------------------------------------------------
// A block's 16 channel rows of one sequence, and a wave's share of their chunks.
struct Channels {
  int j0, n, k0, k1;
  __device__ __forceinline__ Channels(const Product& p, int w) {
    j0 = (int)blockIdx.x * 16;
    n = p.n_dev ? p.n_dev[blockIdx.y] : p.N;
    n = n < p.N ? n : p.N;
    const int chunks = p.pitch / kChunkBytes, per = (chunks + 7) / 8;
    k0 = w * per;
    k1 = k0 + per < chunks ? k0 + per : chunks;
  }
  // the block's channel row r; a hole reads row 0, and nobody reads its output
  __device__ __forceinline__ int id(const Product& p, int r) const {
    const int j = j0 + r < p.N ? j0 + r : p.N - 1;
    const int id = p.ids ? p.ids[(size_t)blockIdx.y * p.N + j] : j;
    return id < 0 || id >= p.V ? 0 : id;
  }
};

constexpr int kRowInLds = kChunkBytes + 16;          // a row's chunk in LDS: 16 rows meet no bank twice

// The eight waves' sums of token operand u joined by wave u.  Lane (i, g) holds
// tokens 4 g .. 4 g + 3 of channel i.
template <int OT, int NMT>
__device__ __forceinline__ void join_waves(const Product& p, f32x4 (&sh)[8][NMT][NS_WAVE], const f32x4 (&acc)[NMT], int w, int lane,
                                           const Channels& c, size_t row0, int M) {
#pragma unroll
  for (int u = 0; u < NMT; ++u) sh[w][u][lane] = acc[u];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < NMT; ++u) {
    if (u != w) continue;
    f32x4 s = sh[0][u][lane];
#pragma unroll
    for (int q = 1; q < 8; ++q) s += sh[q][u][lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = u * 16 + (lane >> 4) * 4 + r, j = c.j0 + (lane & 15);
      if (m < M && j < c.n) store_out<OT>(p.out, (row0 + m) * (size_t)p.sm + (size_t)j * (size_t)p.sn, s[r]);
    }
  }
}

template <int OT, int NMT>
__global__ __launch_bounds__(512) void k_mx4_few(Product p) {
  constexpr int BATCH = NMT <= 2 ? 4 : 2;            // chunks of a row in flight
  __shared__ f32x4 sh[8][NMT][NS_WAVE];
  // a wave's chunk of 16 channel rows and of NMT times 16 token rows
  __shared__ __attribute__((aligned(16))) uint8_t codes[8][NMT + 1][16 * kRowInLds];
  __shared__ __attribute__((aligned(16))) uint8_t scales[8][NMT + 1][16 * kChunkScales];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
  const int m0 = (int)blockIdx.z * NMT * 16, M = p.M - m0, spitch = p.pitch / 16;   // tokens in groups; from here on
  const size_t row0 = (size_t)blockIdx.y * p.M + m0;
  const Channels c(p, w);
  // Eight lanes a row, two loads for 16 rows; of the scales two lanes a row, in
  // either half of the wave.
  const int r8 = lane >> 3, r2 = lane >> 1 & 15;
  const uint8_t *wr[2], *xr[NMT][2], *wsr, *xsr[NMT];
#pragma unroll
  for (int v = 0; v < 2; ++v) wr[v] = p.w + (size_t)c.id(p, v * 8 + r8) * p.pitch + (lane & 7) * 16;
  wsr = p.ws + (size_t)c.id(p, r2) * spitch + (lane & 1) * 4;
#pragma unroll
  for (int u = 0; u < NMT; ++u) {
    const auto row = [&](int r) { return row0 + (u * 16 + r < M ? u * 16 + r : M - 1); };
#pragma unroll
    for (int v = 0; v < 2; ++v) xr[u][v] = p.x + row(v * 8 + r8) * p.pitch + (lane & 7) * 16;
    xsr[u] = p.xs + row(r2) * spitch + (lane & 1) * 4;
  }
  if (c.j0 >= c.n) return;
  f32x4 acc[NMT] = {};
  // `count` chunks at once; those behind the wave's last are its first again, unused
  const auto step = [&](auto count, int k) {
    constexpr int C = decltype(count)::value;
    u32x4 x[C][NMT + 1][2];
    uint32_t s[C][NMT + 1];
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int at = q == 0 || k + q < c.k1 ? k + q : c.k0;
#pragma unroll
      for (int o = 0; o <= NMT; ++o) {
#pragma unroll
        for (int v = 0; v < 2; ++v) x[q][o][v] = *(const u32x4*)((o == 0 ? wr[v] : xr[o > 0 ? o - 1 : 0][v]) + (size_t)at * kChunkBytes);
        s[q][o] = *(const uint32_t*)((o == 0 ? wsr : xsr[o > 0 ? o - 1 : 0]) + at * kChunkScales);
      }
    }
    NS_ISSUE_FENCE();
#pragma unroll
    for (int q = 0; q < C; ++q)
      if (q == 0 || k + q < c.k1) {                  // uniform over the wave
#pragma unroll
        for (int o = 0; o <= NMT; ++o) {
#pragma unroll
          for (int v = 0; v < 2; ++v) *(u32x4*)&codes[w][o][(v * 8 + r8) * kRowInLds + (lane & 7) * 16] = x[q][o][v];
          *(uint32_t*)&scales[w][o][r2 * kChunkScales + (lane & 1) * 4] = s[q][o];
        }
        NS_ISSUE_FENCE();                            // a wave's LDS accesses are in order
        const auto block = [&](int o, int b) { return *(const i32x4*)&codes[w][o][i * kRowInLds + g * 32 + b * 16]; };
        const auto two = [&](int o) { return (uint32_t)*(const uint16_t*)&scales[w][o][i * kChunkScales + g * 2]; };
        const i32x4 a0 = block(0, 0), a1 = block(0, 1);
        const uint32_t sa = two(0);
#pragma unroll
        for (int u = 0; u < NMT; ++u) {
          const uint32_t sb = two(u + 1);
          acc[u] = product128<0>(block(u + 1, 0), a0, acc[u], sb, sa);
          acc[u] = product128<1>(block(u + 1, 1), a1, acc[u], sb, sa);
        }
        NS_ISSUE_FENCE();
      }
  };
  // two or one where no more are left: their loads are not asked for several times
  for (int k = c.k0; k < c.k1; k += BATCH) {
    if (c.k1 - k == 1) step(std::integral_constant<int, 1>(), k);
    else if (BATCH > 2 && c.k1 - k == 2) step(std::integral_constant<int, 2>(), k);
    else step(std::integral_constant<int, BATCH>(), k);
  }
  join_waves<OT>(p, sh, acc, w, lane, c, row0, M);
}

// ---------------------------------------------------------------------------
// The head over few rows with the quantisation of its hidden rows in the same
// launch: each wave quantises the chunks that it multiplies, without a word to
// another.  Half a wave takes a chunk of a row, so that loads are whole lines, and
// the codes pass through LDS to the lanes that multiply them (lanes that read and
// quantised what they multiply asked for 64 lines a load: 8 hidden rows of 4096,
// 1000 channel rows, 8.2 -> 6.5 us).  Bound by latency: the ids, then their rows.
// ---------------------------------------------------------------------------
template <int ET, int NMT>
__global__ __launch_bounds__(512) void k_mx4_head_few(Product p, const void* __restrict__ h, int d) {
  constexpr int ROWS = 8;                            // hidden rows at once, two a load
  __shared__ f32x4 sh[8][NMT][NS_WAVE];
  __shared__ __attribute__((aligned(16))) uint8_t codes[8][NMT * 16 * kRowInLds];
  __shared__ __attribute__((aligned(16))) uint8_t scales[8][NMT * 16 * kChunkScales];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
  const size_t row0 = (size_t)blockIdx.y * p.M;
  const int tail = d & ~(ET == NS_FP32 ? 3 : 7), chunks = p.pitch / kChunkBytes;
  const int l = lane & 31, half = lane >> 5;
  Eight<ET> v[ROWS / 2], next[ROWS / 2];
  // rows m .. m + 7 of chunk k; rows past the last are the last one again
  const auto load = [&](int k, int m, Eight<ET>(&to)[ROWS / 2]) {
#pragma unroll
    for (int t = 0; t < ROWS / 2; ++t) {
      const int r = m + t * 2 + half;
      const char* row = (const char*)h + (row0 + (r < p.M ? r : p.M - 1)) * (size_t)d * (ET == NS_FP32 ? 4 : 2);
      u32x4 rest = {0, 0, 0, 0};
      if (k + 1 == chunks) rest = Eight<ET>::rest_of(row, tail, d);
      to[t].load(row, k * kChunk + l * (ET == NS_FP32 ? 4 : 8), kChunk / 2, tail, rest);
    }
  };
  const Channels c(p, w);
  const int id = c.id(p, i);
  const uint8_t *wr = p.w + (size_t)id * p.pitch + g * 32, *wsr = p.ws + (size_t)id * (p.pitch / 16) + g * 2;
  if (c.k0 < c.k1) load(c.k0, 0, v);
  if (c.j0 >= c.n) return;
  f32x4 acc[NMT] = {};
  for (int k = c.k0; k < c.k1; ++k) {
    const i32x4 a0 = *(const i32x4*)(wr + (size_t)k * kChunkBytes), a1 = *(const i32x4*)(wr + (size_t)k * kChunkBytes + 16);
    const uint32_t sa = *(const uint16_t*)(wsr + k * kChunkScales);
    for (int m = 0; m < p.M; m += ROWS) {
      const bool same = m + ROWS < p.M;
      load(same || k + 1 == c.k1 ? k : k + 1, same ? m + ROWS : 0, next);   // behind the last rows any
      NS_ISSUE_FENCE();
#pragma unroll
      for (int t = 0; t < ROWS / 2; ++t) {
        const int r = m + t * 2 + half;
        put_chunk<ET>(v[t], l, &codes[w][r * kRowInLds], &scales[w][r * kChunkScales]);
      }
#pragma unroll
      for (int t = 0; t < ROWS / 2; ++t) v[t] = next[t];
    }
    NS_ISSUE_FENCE();                                // a wave's LDS accesses are in order
#pragma unroll
    for (int u = 0; u < NMT; ++u) {
      const int r = u * 16 + i;
      const i32x4 b0 = *(const i32x4*)&codes[w][r * kRowInLds + g * 32], b1 = *(const i32x4*)&codes[w][r * kRowInLds + g * 32 + 16];
      const uint32_t sb = *(const uint16_t*)&scales[w][r * kChunkScales + g * 2];
      acc[u] = product128<0>(b0, a0, acc[u], sb, sa);
      acc[u] = product128<1>(b1, a1, acc[u], sb, sa);
    }
    NS_ISSUE_FENCE();
  }
  join_waves<NS_FP32>(p, sh, acc, w, lane, c, row0, p.M);
}

// ---------------------------------------------------------------------------
// The product for up to 64 token rows: bound by the bytes of the channel rows,
// each read once (8 x 128256 x 4096 54 us, 5.2 TB/s; 60 x 151936 x 3584 67 us, 4.6
// TB/s with the outputs; the head's 15500 rows of 4096 for 64 hidden rows 15 us).
//
// One block of eight waves a CU takes an even share of the channel units of ROWS
// rows and runs through it in passes of eight units, one a wave (RT operands of 16
// rows), in stages of one chunk a row.  A ring of stages in LDS is filled by direct
// global-to-LDS loads, R - 1 stages ahead, across the ends of passes; channel
// rows and their scales are private to their wave, token rows shared by the
// block, so one barrier a stage orders the ring; the tokens' scales are in LDS
// from the start.  Waits count the loads that may still be out; outputs leave by
// buffer stores, which out-of-range lanes take part in without effect, so the
// stores behind a pass are as many for every pass and the waits can allow for
// them.
//
// Block b begins every row at chunk 5 b mod S and goes round: blocks that walked
// along their rows in step would read addresses alike in their low bits, a few
// memory channels' worth.
//
// The token rows are operand A and the channel rows operand B, so 16 lanes
// hold 16 consecutive outputs of a token.  Blocks of a row stand in LDS as in
// the tiles below: place c of row r holds block c ^ (r % 8) in that order.
//
// With IDS the channel rows are those that ids names (n_dev of them), the
// block's share of ids waiting in LDS, and blockIdx.y is the sequence.
// ---------------------------------------------------------------------------
constexpr int kStreamWaves = 8;
constexpr int kStreamIds = 4096;                   // ids of a block, at most
constexpr int kStreamIdsD = 8192;                  // d with ids and over 32 tokens, at most: their scales and the ids share what LDS is left

// The 16-byte block of a chunk at place c of a row: 0 2 4 6 1 3 5 7.
__device__ __forceinline__ int block_at(int c) { return (c & 3) * 2 + (c >> 2); }

template <int OT, int NMT, int ROWS, int R, bool IDS>
__global__ __launch_bounds__(kStreamWaves* NS_WAVE, 2) void k_mx4_stream(Product p) {
  constexpr int RT = ROWS > 16 ? ROWS / 16 : 1, PROWS = kStreamWaves * ROWS, LR = ROWS / 8;
  constexpr int XOFF = PROWS * kChunkBytes, SOFF = XOFF + NMT * 16 * kChunkBytes;
  constexpr int STAGE = SOFF + kStreamWaves * 256;   // channel rows, token rows, channel scales
  constexpr int XL = NMT % 4 == 0 ? NMT / 4 : NMT, LW = LR + 1 + XL;   // loads of a wave and stage
  // stores behind a pass that the waits allow for (vmcnt counts to 63)
  constexpr int STORES = RT * NMT * 4 < 63 - (R - 2) * LW ? RT * NMT * 4 : 63 - (R - 2) * LW;
  static_assert((R - 2) * LW + STORES < 64, "vmcnt range");
  constexpr int XS = NMT * 16 * ((IDS && NMT > 2 ? kStreamIdsD : NS_MAX_D) / 32 + 8);   // the tokens' scales, a row's 8 bytes from the next
  __shared__ __attribute__((aligned(16))) char lds[R * STAGE + XS];
  __shared__ int s_id[IDS ? kStreamIds : 1];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
  const int S = p.pitch / kChunkBytes, spitch = S * kChunkScales;
  int live = p.N;
  if (IDS) {
    const size_t seq = blockIdx.y;
    if (p.n_dev) live = p.n_dev[seq];                  // its latency passes under the scales'
    p.x += seq * p.M * p.pitch;
    p.xs += seq * p.M * spitch;
    if (p.ids) p.ids += seq * p.N;
    p.out = (char*)p.out + seq * p.M * (size_t)p.sm * (OT == NS_FP32 ? 4 : 2);
  }
  char* xs = lds + R * STAGE;
  for (int r = tid >> 5; r < NMT * 16; r += kStreamWaves * 2)   // eight scales a lane; rows past the end are the last one's
    for (int c = tid & 31; c < S; c += 32)
      *(u32x2*)(xs + r * (spitch + 8) + c * 8) = *(const u32x2*)(p.xs + (r < p.M ? r : p.M - 1) * spitch + c * 8);
  live = live < 0 ? 0 : (live < p.N ? live : p.N);
  const int units = (live + ROWS - 1) / ROWS, per_block = (units + (int)gridDim.x - 1) / (int)gridDim.x;
  const int u0 = (int)blockIdx.x * per_block, u1 = u0 + per_block < units ? u0 + per_block : units;
  const int passes = (u1 - u0 + kStreamWaves - 1) / kStreamWaves;
  if (passes <= 0) return;
  const uint32_t base = lds_offset(lds);
  const int n0 = u0 * ROWS;                            // the block's first channel row
  const int last = (u1 * ROWS < live ? u1 * ROWS : live) - 1 - n0;
  const u32x4 rw = IDS ? buffer_of(p.w, (uint32_t)p.V * p.pitch)
                       : buffer_of(p.w + (size_t)n0 * p.pitch, (uint32_t)(last + 1) * p.pitch);
  const u32x4 rs = IDS ? buffer_of(p.ws, (uint32_t)p.V * spitch)
                       : buffer_of(p.ws + (size_t)n0 * spitch, (uint32_t)(last + 1) * spitch);
  const u32x4 rx = buffer_of(p.x, (uint32_t)(p.M * p.pitch));
  if (IDS) {                                         // a hole reads row 0; nobody reads its output
    for (int r = tid; r <= last; r += kStreamWaves * NS_WAVE) {
      const int id = p.ids ? p.ids[n0 + r] : n0 + r;
      s_id[r] = id < 0 || id >= p.V ? 0 : id;
    }
  }
  __syncthreads();
  // token rows past the end read the last one and are not stored
  uint32_t xo[XL];
  if (NMT % 4 == 0) {
#pragma unroll
    for (int v = 0; v < XL; ++v) {
      const int r = (v * 8 + w) * 8 + (lane >> 3);
      xo[v] = (uint32_t)((r < p.M ? r : p.M - 1) * p.pitch + block_at((lane & 7) ^ (lane >> 3)) * 16);
    }
  } else {
#pragma unroll
    for (int v = 0; v < NMT; ++v) {                  // two rows a load, a word a lane
      const int r = v * 16 + w * 2 + (lane >> 5), q = lane & 31;
      xo[v] = (uint32_t)((r < p.M ? r : p.M - 1) * p.pitch + block_at((q >> 2) ^ (r & 7)) * 16 + (q & 3) * 4);
    }
  }
  // The stream of loads: the lk-th stage of pass lp comes next, chunk ks of the rows, into place lb.
  const int start = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 5u) % S);
  int lp = 0, lk = 0, lb = 0, ks = start;
  uint32_t wo[LR], so;                           // of the pass
  const auto aim = [&]() {
    const int r0 = (lp * kStreamWaves + w) * ROWS;
    const auto row = [&](int r) {
      r = r < last ? r : last;
      return (uint32_t)(IDS ? s_id[r] : r);
    };
#pragma unroll
    for (int v = 0; v < LR; ++v)
      wo[v] = __umul24(row(r0 + v * 8 + (lane >> 3)), p.pitch) + block_at((lane & 7) ^ (lane >> 3)) * 16;
    so = __umul24(row(r0 + (lane >> 1 & (ROWS - 1))), spitch) + (lane & 1) * 4;
  };
  const auto issue = [&]() {
    const uint32_t to = base + lb * STAGE;
#pragma unroll
    for (int v = 0; v < LR; ++v) load_to_lds_once(rw, wo[v], ks * kChunkBytes, to + (w * LR + v) * 1024);
    load_word_to_lds(rs, so, ks * kChunkScales, to + SOFF + w * 256);
    if (NMT % 4 == 0) {
#pragma unroll
      for (int v = 0; v < XL; ++v) load_to_lds(rx, xo[v], ks * kChunkBytes, to + XOFF + (v * 8 + w) * 1024);
    } else {
#pragma unroll
      for (int v = 0; v < NMT; ++v) load_word_to_lds(rx, xo[v], ks * kChunkBytes, to + XOFF + (v * 8 + w) * 256);
    }
    lb = lb + 1 == R ? 0 : lb + 1;
    ks = ks + 1 == S ? 0 : ks + 1;
    if (++lk == S) {                                 // behind the last pass the stream reads that pass again,
      lk = 0;                                        // which spares every load a question
      if (lp + 1 < passes) {
        ++lp;
        aim();
      }
    }
  };
  aim();
  const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(p.out, 0, 0x7FFFFFFF, 0x00027000);
  constexpr int ESZ = OT == NS_FP32 ? 4 : 2;
  f32x4 acc[RT][NMT] = {};
#pragma unroll
  for (int v = 0; v < R - 1; ++v) issue();
  const int place0 = (g ^ (i & 7)) * 16, place1 = ((4 + g) ^ (i & 7)) * 16;
  const int ir = ROWS < 16 ? i & (ROWS - 1) : i;     // with 8 rows the operand's upper half repeats the lower
  const char* lw = lds + (w * ROWS + ir) * kChunkBytes;
  const char* lx = lds + XOFF + i * kChunkBytes;
  const char* ls = lds + SOFF + w * 256 + ir * kChunkScales + g * 2;
  const char* lxs = xs + i * (spitch + 8) + g * 2;
  int b = 0, since = R, kr = start;                  // stages since the last stores; the chunk that is multiplied
  for (int pass = 0; pass < passes; ++pass) {
    for (int s = 0; s < S; ++s) {
      // this stage's loads are done when at most those of the R - 2 stages
      // behind it, and the stores between them, are out
      if (since < R - 1) wait_loads<(R - 2) * LW + STORES>();
      else wait_loads<(R - 2) * LW>();
      ++since;
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue();                                       // into the place of the stage before, which all have read
      const char* at = lw + b * STAGE;
      const char* xt = lx + b * STAGE;
      i32x4 f[RT][2];
      uint32_t sw[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        sw[t] = *(const uint16_t*)(ls + b * STAGE + t * 16 * kChunkScales);
        f[t][0] = *(const i32x4*)(at + t * 16 * kChunkBytes + place0);
        f[t][1] = *(const i32x4*)(at + t * 16 * kChunkBytes + place1);
      }
#pragma unroll
      for (int u = 0; u < NMT; ++u) {
        const uint32_t sx = *(const uint16_t*)(lxs + u * 16 * (spitch + 8) + kr * kChunkScales);
        const i32x4 x0 = *(const i32x4*)(xt + u * 16 * kChunkBytes + place0);
        const i32x4 x1 = *(const i32x4*)(xt + u * 16 * kChunkBytes + place1);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          acc[t][u] = product128<0>(x0, f[t][0], acc[t][u], sx, sw[t]);
          acc[t][u] = product128<1>(x1, f[t][1], acc[t][u], sx, sw[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < NMT; ++u) asm volatile("" : "+v"(acc[t][u]));   // the products stay in front of the wait
      __builtin_amdgcn_sched_barrier(0);             // no read moves behind the wait
      __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0): this wave has read the stage
      b = b + 1 == R ? 0 : b + 1;
      kr = kr + 1 == S ? 0 : kr + 1;
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int j = (pass * kStreamWaves + w) * ROWS + t * 16 + i;
#pragma unroll
      for (int u = 0; u < NMT; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int m = u * 16 + g * 4 + r;
          const float v = acc[t][u][r];
          const uint32_t to =
              m < p.M && j <= last && (ROWS >= 16 || i < ROWS) ? (uint32_t)(((size_t)m * (size_t)p.sm + (size_t)(n0 + j) * (size_t)p.sn) * ESZ) : 0x80000000u;
          if (OT == NS_FP32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), ro, to, 0, 0);
          else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)narrow2<OT>(v, 0.f), ro, to, 0, 0);
          acc[t][u][r] = 0.f;
        }
    }
    since = 0;
  }
  wait_loads<0>();                                   // the stream's last loads end before their LDS is given back
}

// ---------------------------------------------------------------------------
// The product for many token rows: compute-bound, tiles in LDS.  4096 x 128256 x
// 4096 takes 1000 to 1050 us (4.1 to 4.3 PFLOP/s), 4096 x 16384 x 16384 446 to 486 (4.5 to 4.9).
// The matrix instructions alone reach 7.0 to 7.4 with such data: the power limit
// holds the clock near 1.85 GHz, and they are busy for 59 % of its cycles.  In
// between, a stage's 68 KB come in by direct loads at some 57 bytes a cycle, and
// what the waves read from LDS takes as long as the products.  Stages of half a
// chunk in a deeper ring, loads in other places or in pairs, raised wave priority
// and rows fetched into L2 ahead changed nothing or were slower; reading no scales
// at all would save 3 %.
//
// A block of eight waves owns 256 channel rows and TB * 64 token rows of the
// output; a wave owns 128 channel rows (eight operands of 16) and TB * 16
// token rows (TB operands), 8 TB accumulator tiles in registers.  The sum runs
// in stages of one chunk a row (128 bytes of codes and 8 scales), two in LDS
// (68 KB each with TB = 4), three with TB = 1, whose short stages end before a
// load does, filled by direct global-to-LDS loads.  While one half of a stage (four blocks a
// row) is multiplied, the next half is read into a second set of registers;
// once a wave holds a stage's second half and the next stage has landed, one
// block barrier frees the stage's place for the stage after next.
//
// Blocks stay: each takes one tile after the other, and the stages of all its
// tiles are one stream of loads, so the next tile's first stages arrive while
// the last ones of this tile are multiplied and its outputs are stored.  Tiles
// go to the blocks of one XCD from one contiguous run, in groups of four channel
// tiles by all token tiles, so that its 32 CUs share rows in its L2.
//
// Lane i of channel operand t is channel row 8 i + t, so the eight
// accumulators of a lane are eight consecutive outputs and a store of 16
// lanes covers 128 of them, without a detour through LDS.  Lane (i, g) takes
// blocks 2 g and 2 g + 1 of a chunk, whose two scales are one 16-bit read.
//
// The eight 16-byte blocks of a row stand in LDS with the four even ones (those of
// the first half) first; place c of row r holds the one that is c ^ (r / 8 % 8)
// in that order in channel rows and c ^ (r % 8) in token rows, and eight channel
// rows stand 128 bytes from the next eight, so that lanes i and i + 1 read from
// different halves of the 64 banks: no bank is met twice.  Scales stand in the
// order in which the lanes read them, 16 bytes a row for two stages; a bank is met
// twice there (reads without that took the same time, 1030 and 1031 us).
// ---------------------------------------------------------------------------
constexpr int kTileN = 256;                        // channel rows of a block
constexpr int kTileThreads = 512;
constexpr int tile_stages(int tb) { return tb == 1 ? 3 : 2; }   // in LDS
constexpr int kEightRows = 9 * kChunkBytes;        // eight channel rows in LDS and 128 bytes between them and the next

// Eight consecutive 16-bit outputs, aligned, that nobody reads soon.
template <int OT>
__device__ __forceinline__ void store_once(void* out, size_t i, const float (&v)[8]) {
  __builtin_nontemporal_store(u32x4{narrow2<OT>(v[0], v[1]), narrow2<OT>(v[2], v[3]), narrow2<OT>(v[4], v[5]), narrow2<OT>(v[6], v[7])},
                              (u32x4*)((uint16_t*)out + i));
}

template <int OT, int TB>
__global__ __launch_bounds__(kTileThreads, 2) void k_mx4_tiled(Product p, int tiles_m, int tiles_n) {
  constexpr int TM = TB * 64;                      // token rows of a block
  constexpr int XOFF = kTileN / 8 * kEightRows, STAGE = XOFF + TM * kChunkBytes;
  constexpr int LA = kTileN / 64, LB = TM / 64;    // loads of a wave and stage: 8 rows each
  constexpr int STORES = TB * 4 * (OT == NS_FP32 ? 2 : 1);   // of a wave and whole tile
  constexpr int R = tile_stages(TB), AHEAD = (R - 2) * (LA + LB);   // loads that may be out when a stage must be here
  static_assert(AHEAD + STORES < 64, "vmcnt range");
  // scales of two stages together, R such pairs
  constexpr int SOFF = R * STAGE, PAIR = (kTileN + TM) * 2 * kChunkScales;
  __shared__ __attribute__((aligned(16))) char lds[SOFF + R * PAIR];
  const int total = tiles_m * tiles_n, per = (total + 7) / 8, slots = (int)(gridDim.x >> 3);
  const int first = (int)(blockIdx.x & 7) * per, end = first + per < total ? first + per : total;
  int tile = first + (int)(blockIdx.x >> 3);
  if (tile >= end) return;
  const auto origin = [&](int t, int& m0, int& n0) {
    const int group = t / (tiles_m * 4), rest = t % (tiles_m * 4);
    const int wide = tiles_n - group * 4 < 4 ? tiles_n - group * 4 : 4;   // channel tiles of this group
    n0 = (group * 4 + rest % wide) * kTileN;
    m0 = rest / wide * TM;
  };
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
  const int S = p.pitch / kChunkBytes, spitch = p.pitch / 16;
  const uint32_t base = lds_offset(lds);

  // The stream of loads: stage `lk` of tile `lt` comes next.
  int lt = tile, lk = 0, lp = 0;
  u32x4 ra, rb, rs;
  int last_a, last_b;                              // rows past the end read the last one and are not stored
  uint32_t at[LA + LB];                            // of the tile's loads
  const int tw = (w & 3) % TB;                     // scales: waves 0 to 3 the channels', 4 to 7 the tokens', 64 rows each
  const auto aim = [&]() {
    int m0, n0;
    origin(lt, m0, n0);
    last_a = p.N - 1 - n0;
    last_b = p.M - 1 - m0;
    ra = buffer_of(p.w + (size_t)n0 * p.pitch, (uint32_t)(kTileN * p.pitch));
    rb = buffer_of(p.x + (size_t)m0 * p.pitch, (uint32_t)(TM * p.pitch));
#pragma unroll
    for (int u = 0; u < LA + LB; ++u) {
      const int v = u < LA ? u : u - LA, r = (v * 8 + w) * 8 + (lane >> 3), last = u < LA ? last_a : last_b;
      at[u] = __umul24(r < last ? r : last, p.pitch) + block_at((lane & 7) ^ (u < LA ? w : lane >> 3)) * 16;
    }
    // the range ends with the rows: behind the last one's scales there may be nothing to read
    rs = w < 4 ? buffer_of(p.ws + (size_t)n0 * spitch, (uint32_t)((last_a < kTileN ? last_a + 1 : kTileN) * spitch))
               : buffer_of(p.xs + (size_t)m0 * spitch, (uint32_t)((last_b < TM ? last_b + 1 : TM) * spitch));
  };
  // Load u of the next stage's LA + LB, into buffer buf.
  const auto load = [&](int u, int buf) {
    const int v = u < LA ? u : u - LA;
    load_to_lds(u < LA ? ra : rb, at[u], lk * kChunkBytes,
                base + buf * STAGE + (u < LA ? (v * 8 + w) * kEightRows : XOFF + (v * 8 + w) * 8 * kChunkBytes));
  };
  // Behind an even stage's loads the scales of that stage and the next, a row a
  // lane (a row's 16 bytes at once: with 4 a lane for each stage the loads, 64
  // lines of memory each, took 230 of 1240 us), then on to the next stage.
  const auto advance = [&]() {
    if ((lk & 1) == 0) {
      int l = lane;
      asm volatile("" : "+v"(l));
      // place t * 16 + i of a wave's 128 channel rows holds row 8 i + t
      const int q = (w & 3) * 64 + l, r = w < 4 ? (q & 128) + (q & 15) * 8 + (q >> 4 & 7) : tw * 64 + l;
      const int last = w < 4 ? last_a : last_b;
      load_to_lds(rs, __umul24(r < last ? r : last, spitch), lk * kChunkScales,
                  base + SOFF + lp * PAIR + (w < 4 ? w : 4 + tw) * 1024);
      lp = lp + 1 == R ? 0 : lp + 1;
    }
    if (++lk == S) {                               // behind the last tile the stream reads that tile again,
      lk = 0;                                      // which spares every load a question
      if (lt + slots < end) {
        lt += slots;
        aim();
      }
    }
  };

  const int wr = w >> 2, wc = w & 3;
  f32x4 acc[8][TB] = {};
  // The channel operands of the half that is multiplied, 6 and 7 apart: the
  // next half's replace 0 to 5 as they fall free, and 6 and 7 alternate, so
  // that no read is still to come behind the half's last products.
  i32x4 fa[6], fe[2][2], fb[2][TB];
  // Scales of the stage that is multiplied; the next stage's replace the channels'
  // as they fall free.
  u16x2 sa[8], sb[TB], nb[TB];
  // operand t: channel rows wr * 128 + 8 i + t; operand u: token rows (wc * TB + u) * 16 + i
  const char* la = lds + (wr * 16 + i) * kEightRows;
  const char* lb = lds + XOFF + (wc * TB * 16 + i) * kChunkBytes;
  const char* lsa = lds + SOFF + (wr * 128 + i) * 2 * kChunkScales + g * 2;
  const char* lsb = lds + SOFF + (kTileN + wc * TB * 16 + i) * 2 * kChunkScales + g * 2;
  const int place0 = (g ^ (i & 7)) * 16, place1 = ((4 + g) ^ (i & 7)) * 16;
  // from byte `at` of the pairs
  const auto channel_scales = [&](int t, int at) {
    sa[t] = two_scales(lsa + at + t * 32 * kChunkScales);
  };
  const auto token_scales = [&](int at) {
#pragma unroll
    for (int u = 0; u < TB; ++u) nb[u] = two_scales(lsb + at + u * 32 * kChunkScales);
  };
  aim();
#pragma unroll
  for (int buf = 0; buf < R; ++buf) {
#pragma unroll
    for (int u = 0; u < LA + LB; ++u) load(u, buf);
    advance();
  }
  wait_loads<AHEAD + LA + LB>();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  token_scales(0);
#pragma unroll
  for (int u = 0; u < TB; ++u) sb[u] = nb[u];
#pragma unroll
  for (int t = 0; t < 8; ++t) channel_scales(t, 0);
#pragma unroll
  for (int u = 0; u < TB; ++u) fb[0][u] = *(const i32x4*)(lb + place0 + u * 16 * kChunkBytes);
#pragma unroll
  for (int t = 0; t < 6; ++t) fa[t] = *(const i32x4*)(la + place0 + t * kChunkBytes);
  fe[0][0] = *(const i32x4*)(la + place0 + 6 * kChunkBytes);
  fe[0][1] = *(const i32x4*)(la + place0 + 7 * kChunkBytes);
  // Multiplies the half F in registers (fe, fb of F) and reads the next from
  // `at`.  With F = 1 the next stage's loads go out between the products, one
  // for each operand, and the scales at `from` are read.
  const auto step = [&](auto half, int at, int buf, int from) {
    constexpr int F = decltype(half)::value;
    if (F == 1) token_scales(from);
#pragma unroll
    for (int u = 0; u < TB; ++u) fb[1 - F][u] = *(const i32x4*)(lb + at + u * 16 * kChunkBytes);
    uint32_t st[TB];
#pragma unroll
    for (int u = 0; u < TB; ++u) st[u] = __builtin_bit_cast(uint32_t, sb[u]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (F == 1 && t < LA + LB) load(t, buf);
      const i32x4 a = t < 6 ? fa[t % 6] : fe[F][t & 1];
      const uint32_t sc = __builtin_bit_cast(uint32_t, sa[t]);
#pragma unroll
      for (int u = 0; u < TB; ++u) {
        acc[t][u] = product128<F>(fb[F][u], a, acc[t][u], st[u], sc);
        asm volatile("" : "+v"(acc[t][u]));        // the product stays here, between the loads
      }
      if (t < 6) fa[t % 6] = *(const i32x4*)(la + at + t * kChunkBytes);
      if (t == 3 || t == 4) fe[1 - F][t - 3] = *(const i32x4*)(la + at + (t + 3) * kChunkBytes);
      if (F == 1) channel_scales(t, from);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int b = 0, pair = 0;
  bool stored = false;                             // the tile before was whole: STORES stores are behind the loads
  for (; tile < end; tile += slots) {
    for (int s = 0; s < S; ++s) {
      step(std::integral_constant<int, 0>(), b * STAGE + place1, 0, 0);
      __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0): this wave has read the stage
      if (s == 0 && stored) wait_loads<AHEAD + STORES>();
      else wait_loads<AHEAD>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      const int next = b + 1 == R ? 0 : b + 1;
      const int s1 = s + 1 == S ? 0 : s + 1;       // the next stage's number
      if ((s1 & 1) == 0) pair = pair + 1 == R ? 0 : pair + 1;
      step(std::integral_constant<int, 1>(), next * STAGE + place0, b, pair * PAIR + (s1 & 1) * kChunkScales);
#pragma unroll
      for (int u = 0; u < TB; ++u) sb[u] = nb[u];
      advance();
      b = next;
    }
    int m0, n0, l = lane;
    asm volatile("" : "+v"(l));                    // as in load
    const int ni = (l & 15) * 8, mg = (l >> 4) * 4;
    origin(tile, m0, n0);
    const int n = n0 + wr * 128 + ni;
    stored = m0 + TM <= p.M && n0 + kTileN <= p.N;
    // Whole lines past the caches (4096 x 128256 x 4096 1022 -> 996 us); parts of
    // lines would be written one by one (4096 x 30001 x 512 68 -> 143).
    const bool lines = OT != NS_FP32 && stored && ((uint64_t)p.out | (uint64_t)p.sm * 2) % 128 == 0;
#pragma unroll
    for (int u = 0; u < TB; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = m0 + (wc * TB + u) * 16 + mg + r;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[e][u][r];
        const size_t at = (size_t)m * (size_t)p.sm + n;
        if (lines) store_once<OT>(p.out, at, v);
        else if (m < p.M && n < p.N) store_eight<OT>(p.out, at, v, p.N - n);
      }
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int u = 0; u < TB; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  wait_loads<0>();                                 // the stream's last loads end before their LDS is given back
}

template <int OT, int TB>
void launch_tiled(const Product& p, hipStream_t stream) {
  const int tm = (p.M + TB * 64 - 1) / (TB * 64), tn = (p.N + kTileN - 1) / kTileN;
  // one block a CU, eight XCDs of 32 CUs
  const unsigned per = ((unsigned)tm * (unsigned)tn + 7) / 8;
  hipLaunchKernelGGL((k_mx4_tiled<OT, TB>), dim3((per < 32 ? per : 32) * 8), dim3(kTileThreads), 0, stream, p, tm, tn);
}

template <int OT, int NMT>
void launch_few(const Product& p, int B, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)B, (unsigned)((p.M + NMT * 16 - 1) / (NMT * 16)));
  hipLaunchKernelGGL((k_mx4_few<OT, NMT>), grid, dim3(512), 0, stream, p);
}

template <int OT>
void launch_few_of(const Product& p, int B, hipStream_t stream) {
  if (p.M <= 16) launch_few<OT, 1>(p, B, stream);
  else if (p.M <= 32) launch_few<OT, 2>(p, B, stream);
  else if (p.M <= 48) launch_few<OT, 3>(p, B, stream);
  else launch_few<OT, 4>(p, B, stream);
}

template <int OT, int NMT, int ROWS, int R>
void launch_stream(const Product& p, hipStream_t stream) {
  const int units = (p.N + ROWS - 1) / ROWS, per = (units + 255) / 256;
  hipLaunchKernelGGL((k_mx4_stream<OT, NMT, ROWS, R, false>), dim3((unsigned)((units + per - 1) / per)),
                     dim3(kStreamWaves * NS_WAVE), 0, stream, p);
}

// The kernel for few rows is taken up to this many of its blocks of 16 channels and (up to) 64 tokens.  Against the
// stream: up to 16 tokens four a CU (d = 4096, M = 8: 12000 channels 7.0 us against 9.1, 16000 8.7 against 10.4), three
// where rows are short (d = 256: 12000 3.8 and 3.7, 16000 4.2 against 3.7); up to 48 tokens two (M = 32, 8000 channels:
// d = 4096 8.0 against 10.1, d = 256 4.1 and 4.2); up to 64 two from d = 1024 to 4096 (8000 channels: d = 256 5.5
// against 5.0, 1024 6.5 and 6.4, 4096 11.8 and 12.3, 8192 20.7 against 19.0).  Against tiles: one a CU (1000 x 256 x
// 4096 7.0 against 13.0, x 256 3.6 against 4.7), and two where rows are long and of tokens not many, whose rows each
// channel block asks for anew (400 x 1000 x 256 5.6 against 5.2, x 1024 6.6 and 6.5, x 2048 8.5 against 8.9, x 4096 12.1
// against 13.5; 2000 x 250 x 4096 12.9 against 14.1, 3000 x 160 x 4096 13.9 and 13.6, 4096 x 100 x 4096 15.0 against
// 13.6); not four (1000 x 1000 x 4096 23.5 against 13.6).
int few_blocks(int M, int d) {
  if (M <= 16) return d >= 1024 ? 1024 : 768;
  if (M <= 48) return 512;
  if (M <= 64) return d >= 1024 && d <= 4096 ? 512 : 256;
  return d >= 2048 && M <= 2048 ? 512 : 256;
}

// Up to 64 tokens what the kernel for few rows leaves takes the stream, of eight-row units up to 16384 channels (M =
// 64, 16000 13.5 against 16.1 with taller units; 60 x 30000 x 3584 20.7 against 18.7) and for up to 16 tokens (M = 8,
// 30000 15.0 against 17.0, 128256 57.4 against 58.6).
// The rest takes tiles of 256, 128 or 64 tokens.  Blocks take one tile each a
// round, and a round takes about 28, 21 and 17 us at d = 4096 (256 x 16384, one
// round each: 27.2, 20.9, 18.3); the sum over the rounds decides (1000 x 8000 x
// 4096, rounds 1, 1 and 2: 30.1, 25.2, 31.9; 128 x 128256 x 4096, rounds 2, 2 and 4:
// 75.5, 67.0, 78.6).
template <int OT>
void launch_product(const Product& p, hipStream_t stream) {
  const uint64_t span = ((uint64_t)(p.M - 1) * (uint64_t)p.sm + (uint64_t)(p.N - 1) * (uint64_t)p.sn + 1) *
                        (OT == NS_FP32 ? 4 : 2);
  const int64_t few = (int64_t)((p.N + 15) / 16) * ((p.M + 63) / 64);   // blocks of the kernel for few rows
  if (few <= few_blocks(p.M, p.pitch * 2) || (p.M <= 64 && span >= 0x7FFFFFFFull)) {   // the stream's output offsets have 31 bits
    launch_few_of<OT>(p, 1, stream);
  } else if (p.M <= 64) {
    if (p.M <= 16) {
      launch_stream<OT, 1, 8, 7>(p, stream);
    } else if (p.N <= 16384) {
      if (p.M <= 32) launch_stream<OT, 2, 8, 7>(p, stream);
      else if (p.M <= 48) launch_stream<OT, 3, 8, 7>(p, stream);
      else launch_stream<OT, 4, 8, 7>(p, stream);
    } else {
      if (p.M <= 32) launch_stream<OT, 2, 16, 6>(p, stream);
      else if (p.M <= 48) launch_stream<OT, 3, 32, 3>(p, stream);
      else launch_stream<OT, 4, 32, 3>(p, stream);
    }
  } else {
    const auto time = [&](int tb, int round) {
      const int64_t tiles = (int64_t)((p.N + kTileN - 1) / kTileN) * ((p.M + tb * 64 - 1) / (tb * 64));
      return (tiles + 255) / 256 * round;
    };
    const int64_t t4 = time(4, 28), t2 = time(2, 21), t1 = time(1, 17);
    if (t4 <= t2 && t4 <= t1) launch_tiled<OT, 4>(p, stream);
    else if (t2 <= t1) launch_tiled<OT, 2>(p, stream);
    else launch_tiled<OT, 1>(p, stream);
  }
}

template <int NMT, int ROWS, int R>
void launch_head_stream(const Product& p, int B, hipStream_t stream) {
  // one block a CU over all sequences, none with more ids than it holds
  const int units = (p.N + ROWS - 1) / ROWS, least = (units * ROWS + kStreamIds - 1) / kStreamIds;
  int gx = B < 256 ? 256 / B : 1;
  gx = gx > units ? units : (gx < least ? least : gx);
  hipLaunchKernelGGL((k_mx4_stream<NS_FP32, NMT, ROWS, R, true>), dim3((unsigned)gx, (unsigned)B),
                     dim3(kStreamWaves * NS_WAVE), 0, stream, p);
}

// The head's logits, B sequences.  Whole calls (d = 4096), the kernel for few rows
// against the stream: M = 8, 16000 rows 18.0 against 19.6 us; M = 32, 8000 17.1 against
// 19.7, 16000 24.1 against 21.7; M = 64, 8000 21.3 against 21.8.  Eight-row units
// against taller ones: M = 64, 15500 rows 24.6 against 27.5, 100000 81.1 against 68.8;
// M = 8, 100000 59.5 against 60.7.  The stream's 32-bit row addresses reach 4 GB.
bool few_rows(int B, int n_max, int V, int M, int d) {
  return (int64_t)B * n_max <= (M <= 16 ? 16384 : 8192) || (M > 32 && d > kStreamIdsD) || (uint64_t)V * (uint64_t)pitch_of(d) > 0xFFFFFFFFull;
}

// Whether the kernel for few rows also quantises, which each of its blocks does
// again: by how often a wave does so (`work`: eight rows of a chunk each) and by the
// blocks a CU.  One launch less: bf16, d = 4096, M = 8, 4000 rows 11.7 us, 8000 14.7
// and 14.8 in two launches, 16000 22.9 and 18.0; M = 16, 4000 13.0 and 14.5, 8000 18.3
// and 14.6; M = 32, 1000 16.8 and 14.5; d = 1024, M = 8, 16000 14.1 and 14.6.  float32
// rows are twice the loads: M = 24, d = 2048, 1000 rows 13.1 and 14.1; M = 32 14.7 and
// 14.2.
bool fuses_rows(int B, int n_max, int M, int d, int dtype) {
  const int work = (M + 7) / 8 * ((chunks_of(d) + 7) / 8), most = dtype == NS_FP32 ? 8192 : 16384;
  return work <= (dtype == NS_FP32 ? 3 : 4) && (int64_t)B * n_max * work <= most;
}

template <int ET>
void launch_fused(const Product& p, int B, const void* h, int d, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)B), block(512);
  if (p.M <= 16) hipLaunchKernelGGL((k_mx4_head_few<ET, 1>), grid, block, 0, stream, p, h, d);
  else hipLaunchKernelGGL((k_mx4_head_few<ET, 2>), grid, block, 0, stream, p, h, d);   // no more than 32
}

void launch_head(const Product& p, int B, int d, hipStream_t stream) {
  if (few_rows(B, p.N, p.V, p.M, d)) {
    launch_few_of<NS_FP32>(p, B, stream);
  } else if (p.M <= 16) {
    launch_head_stream<1, 8, 7>(p, B, stream);
  } else if ((int64_t)B * p.N <= 16384) {
    if (p.M <= 32) launch_head_stream<2, 8, 7>(p, B, stream);
    else if (p.M <= 48) launch_head_stream<3, 8, 7>(p, B, stream);
    else launch_head_stream<4, 8, 7>(p, B, stream);
  } else {
    if (p.M <= 32) launch_head_stream<2, 16, 5>(p, B, stream);
    else if (p.M <= 48) launch_head_stream<3, 32, 3>(p, B, stream);
    else launch_head_stream<4, 32, 3>(p, B, stream);
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace of the restricted head: the quantised hidden rows and their
// scales, the logits, and the chunks' keys.
struct HeadWs {
  size_t q, scale, z, cand, bytes;
  int64_t ld;
  int chunks;
};

HeadWs head_ws(int B, int n_max, int M, int k, int d) {
  HeadWs w;
  w.ld = ((int64_t)n_max + 3) / 4 * 4;
  w.chunks = (n_max + top_chunk(n_max) - 1) / top_chunk(n_max);
  const size_t rows = (size_t)B * M;
  w.q = 0;
  w.scale = w.q + align256(rows * pitch_of(d));
  w.z = w.scale + align256(rows * (pitch_of(d) / 16));
  w.cand = w.z + align256(rows * (size_t)w.ld * 4);
  w.bytes = w.cand + (w.chunks > 1 ? align256(rows * w.chunks * (size_t)k * 8) : 0);
  return w;
}

constexpr int64_t kMaxLd = (int64_t)1 << 40;       // no product with a row count overflows

bool known_dtype(int t) { return t == NS_BF16 || t == NS_FP32 || t == NS_FP16; }
bool aligned(const void* p, int to) { return (((uintptr_t)p) & (uintptr_t)(to - 1)) == 0; }
bool elem_aligned(const void* p, int dtype) { return aligned(p, dtype == NS_FP32 ? 4 : 2); }
// Codes are read 16 bytes at a time, scales up to eight.
bool rows_aligned(const void* q, const void* scale) { return aligned(q, 16) && aligned(scale, 8); }

bool head_dims_ok(int B, int n_max, int M, int k, int d) {
  return B >= 1 && B <= NS_MAX_BATCH && n_max >= 1 && n_max <= NS_MAX_V && M >= 1 && M <= NS_MAX_M && k >= 1 &&
         k <= NS_MAX_K && d >= 1 && d <= NS_MAX_D;
}

}  // namespace

extern "C" {

int32_t nanospec_mx4_pitch(int32_t d) { return d < 1 || d > NS_MAX_D ? 0 : pitch_of(d); }

int nanospec_mx4_rows(const void* x, int64_t ld, int32_t R, int32_t d, int32_t dtype, uint8_t* q, uint8_t* scale,
                      hipStream_t stream) {
  if (!known_dtype(dtype)) return NS_EDTYPE;
  if (R < 0 || R > NS_MAX_ROWS || d < 1 || d > NS_MAX_D || ld < d || ld > kMaxLd) return NS_EINVAL;
  if (R == 0) return NS_OK;
  if (!x || !q || !scale || !rows_aligned(q, scale) || !elem_aligned(x, dtype)) return NS_EINVAL;
  (void)hipGetLastError();
  return mx4_rows(x, ld, R, d, dtype, q, scale, stream);
}

int nanospec_mx4_gather_rows(const uint8_t* q, const uint8_t* scale, int32_t V, int32_t d, const int32_t* ids,
                             const int32_t* n_dev, int32_t n_max, void* out, int64_t ld_out, int32_t out_dtype,
                             hipStream_t stream) {
  if (!known_dtype(out_dtype)) return NS_EDTYPE;
  if (V < 1 || V > NS_MAX_V || n_max < 0 || n_max > NS_MAX_ROWS || (!ids && n_max > V) || d < 1 || d > NS_MAX_D ||
      ld_out < d || ld_out > kMaxLd)
    return NS_EINVAL;
  if (n_max == 0) return NS_OK;
  if (!q || !scale || !out || !rows_aligned(q, scale) || !elem_aligned(out, out_dtype)) return NS_EINVAL;
  (void)hipGetLastError();
  if (out_dtype == NS_BF16) launch_gather<NS_BF16>(q, scale, V, d, ids, n_dev, n_max, out, ld_out, stream);
  else if (out_dtype == NS_FP16) launch_gather<NS_FP16>(q, scale, V, d, ids, n_dev, n_max, out, ld_out, stream);
  else launch_gather<NS_FP32>(q, scale, V, d, ids, n_dev, n_max, out, ld_out, stream);
  return ns_launch_status();
}

int nanospec_mx4_matmul(const uint8_t* xq, const uint8_t* xs, int32_t M, const uint8_t* wq, const uint8_t* ws, int32_t N,
                        int32_t d, void* out, int64_t ld_out, int32_t out_dtype, hipStream_t stream) {
  if (!known_dtype(out_dtype)) return NS_EDTYPE;
  if (M < 0 || M > NS_MAX_ROWS || N < 1 || N > NS_MAX_V || d < 1 || d > NS_MAX_D || ld_out < N ||
      ld_out > kMaxLd)
    return NS_EINVAL;
  if (M == 0) return NS_OK;
  if (!xq || !xs || !wq || !ws || !out || !rows_aligned(xq, xs) || !rows_aligned(wq, ws)) return NS_EINVAL;
  if (!elem_aligned(out, out_dtype)) return NS_EINVAL;
  (void)hipGetLastError();
  const Product p{xq, xs, wq, ws, nullptr, nullptr, M, N, N, pitch_of(d), out, ld_out, 1};
  if (out_dtype == NS_FP32) launch_product<NS_FP32>(p, stream);
  else if (out_dtype == NS_BF16) launch_product<NS_BF16>(p, stream);
  else launch_product<NS_FP16>(p, stream);
  return ns_launch_status();
}

size_t nanospec_mx4_logits_workspace_bytes(int32_t B, int32_t n_max, int32_t M, int32_t k, int32_t d) {
  return head_dims_ok(B, n_max, M, k, d) ? head_ws(B, n_max, M, k, d).bytes : 0;
}

int nanospec_mx4_logits_topk(const uint8_t* wq, const uint8_t* wscale, const int32_t* row_ids, const int32_t* n_dev,
                             int32_t n_max, int32_t B, int32_t V, int32_t d, const void* h, int32_t dtype, int32_t M,
                             int32_t k, float* logits, int32_t* topk_ids, float* topk_vals, void* ws,
                             size_t ws_bytes, hipStream_t stream) {
  if (!known_dtype(dtype)) return NS_EDTYPE;
  if (!head_dims_ok(B, n_max, M, k, d) || V < 1 || V > NS_MAX_V || (!row_ids && n_max > V)) return NS_EINVAL;
  if (!wq || !wscale || !h || !topk_ids || !topk_vals || !ws) return NS_EINVAL;
  if (!rows_aligned(wq, wscale) || !aligned(ws, 256) || !elem_aligned(h, dtype)) return NS_EINVAL;
  const HeadWs l = head_ws(B, n_max, M, k, d);
  if (ws_bytes < l.bytes) return NS_ECAPACITY;
  (void)hipGetLastError();
  char* base = (char*)ws;
  uint8_t* hq = (uint8_t*)(base + l.q);
  uint8_t* hs = (uint8_t*)(base + l.scale);
  float* z = (float*)(base + l.z);
  const Product p{hq, hs, wq, wscale, row_ids, n_dev, M, n_max, V, pitch_of(d), z, l.ld, 1};
  int rc;
  if (fuses_rows(B, n_max, M, d, dtype)) {
    if (dtype == NS_BF16) launch_fused<NS_BF16>(p, B, h, d, stream);
    else if (dtype == NS_FP16) launch_fused<NS_FP16>(p, B, h, d, stream);
    else launch_fused<NS_FP32>(p, B, h, d, stream);
  } else {
    rc = mx4_rows(h, d, B * M, d, dtype, hq, hs, stream);
    if (rc != NS_OK) return rc;
    launch_head(p, B, d, stream);
  }
  rc = ns_launch_status();
  if (rc != NS_OK) return rc;
  const Top t{z, l.ld, row_ids, n_dev, n_max, V, M, k, logits, topk_ids, topk_vals, (uint64_t*)(base + l.cand)};
  return launch_top(t, l.chunks, B, stream);
}

}  // extern "C"
