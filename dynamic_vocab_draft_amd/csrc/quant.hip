// 8-bit rows: quantisation, the integer product, and the restricted LM head
// over 8-bit rows.
//
// A row x of d elements becomes d 8-bit integers and one float32 scale,
//     a = max |x_i|,  s = a / 127,  q_i = round(127 x_i / a)  (halves to even),
// and the product of a token row and a channel row is
//     out[m, n] = (sum_i xq[m, i] wq[n, i]) * (xs[m] * ws[n]).
// The integer sum is exact: |q| <= 128 and d <= 16384 keep it within 2^28,
// inside the int32 accumulators of v_mfma_i32_16x16x64_i8.  It is rounded
// once to float32, multiplied by the float32 product of the two scales, and
// rounded once to the output type, so results do not depend on how the sum
// was split, and two runs agree bit for bit.
#include "common.hpp"
#include "select.hpp"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kPitch = 128;            // 8-bit rows start every multiple of 128 bytes
__host__ __device__ constexpr int pitch_of(int d) { return (d + kPitch - 1) / kPitch * kPitch; }

// ---------------------------------------------------------------------------
// Row quantisation: one pass, bound by its bytes.  The lanes of a row hold it in
// registers (up to eight groups of eight elements each) between the maximum and
// the rounding (128256 x 4096 bf16 269 us, 5.9 TB/s read and written; 30000 x
// 4096 float32 99 us, 6.2).
// ---------------------------------------------------------------------------
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // rows start at any element
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <int ET>
__device__ __forceinline__ uint32_t load_bits(const void* x, size_t i) {
  return ET == NS_FP32 ? ((const uint32_t*)x)[i] : ((const uint16_t*)x)[i];
}

// Eight elements as they are stored: 16-bit types in one vector, float32 in two.
template <int ET>
struct Eight {
  u32x4 v[ET == NS_FP32 ? 2 : 1];

  // elements i .. i + 7 of a row, or i .. i + 3 and `step` on, zeros at or past
  // d.  `tail` is d rounded down to a vector's elements, `rest` what follows in
  // the row.  The loads stand under no condition that differs from lane to lane.
  __device__ __forceinline__ void load(const char* row, int i, int step, int tail, u32x4 rest) {
    constexpr int N = ET == NS_FP32 ? 2 : 1;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int at = i + n * step;
      u32x4 x = {0, 0, 0, 0};
      if (tail > 0) x = __builtin_nontemporal_load((const u32x4_any*)(row + (size_t)(at < tail ? at : 0) * (2 * N)));
      v[n] = at < tail ? x : (at == tail ? rest : u32x4{0, 0, 0, 0});
    }
  }
  // Elements tail .. d - 1, fewer than a vector's, and zeros.
  static __device__ __forceinline__ u32x4 rest_of(const char* row, int tail, int d) {
    u32x4 r = {0, 0, 0, 0};
    if (tail < d) {                                // uniform
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (ET == NS_FP32) {
          if (tail + c < d) r[c] = load_bits<ET>(row, tail + c);
        } else {
          if (tail + c * 2 < d) r[c] = load_bits<ET>(row, tail + c * 2);
          if (tail + c * 2 + 1 < d) r[c] |= load_bits<ET>(row, tail + c * 2 + 1) << 16;
        }
      }
    }
    return r;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (ET == NS_FP32) return __uint_as_float(v[e >> 2][e & 3]);
    else if constexpr (ET == NS_BF16) return e & 1 ? ns::bf16_hi(v[0][e >> 1]) : ns::bf16_lo(v[0][e >> 1]);
    else return e & 1 ? ns::fp16_hi(v[0][e >> 1]) : ns::fp16_lo(v[0][e >> 1]);
  }
  // The largest magnitude as the type's own bits, which order like the values
  // with infinities and NaN on top; two at once for 16-bit types.
  __device__ __forceinline__ uint32_t top(uint32_t so_far) const {
    if constexpr (ET == NS_FP32) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t u = v[n][c] & 0x7FFFFFFFu;
          so_far = u > so_far ? u : so_far;
        }
      return so_far;
    } else {
      u16x2 m = __builtin_bit_cast(u16x2, so_far);
#pragma unroll
      for (int c = 0; c < 4; ++c) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[0][c] & 0x7FFF7FFFu));
      return __builtin_bit_cast(uint32_t, m);
    }
  }
};

// How a row is quantised: 0 for one of zeros or with a value that is not
// finite (q = 0), otherwise values times `up`, a = up max |x|, rcp = 1 / a.
// `up` brings the maximum into [2^-100, 2^100], where 1 / a and 127 a are far
// from overflow; it is exact for all that is not far below the maximum.
struct Scaling {
  float up, a, rcp;
  bool ok;
  __device__ __forceinline__ explicit Scaling(uint32_t m) {   // the maximum's float32 bits
    const float top = __uint_as_float(m);
    ok = m != 0 && m < 0x7F800000u;
    up = top < 0x1p-100f ? 0x1p64f : (top > 0x1p100f ? 0x1p-64f : 1.f);
    a = top * up;
    rcp = 1.f / a;
  }
};

// Eight elements to eight bytes, round(127 x / a), halves to even, decided
// exactly and without a branch.  Adding 1.5 * 2^23 leaves a value rounded to an
// integer, halves to even, in the low byte.
// 16-bit types: q = 127 x * rcp is off by 2^-23 relatively at most, its
// remainder 127 x - q a is exact (one fused multiply-add of terms with at most
// 18 bits and 24 + 11), and q + remainder * rcp is then the quotient rounded
// to float32: a half comes out as itself, and whatever lies beside one by at
// least 2^-20 of its size (254 x and an odd multiple of a differ by a unit of
// x or a) stays on its side.
// float32: 127 x = m + rest exactly in two floats.  n, m * rcp rounded to an
// integer, is the quotient's rounding or, next to a half, perhaps the integer
// beyond; r = m - n a is exact, and so is |r| - a / 2 next to a half, so `over`
// has the sign of the true remainder's excess over a / 2: above 0, or 0 with n
// odd (no float but 0 is below the smallest positive one), n moves by one
// towards r.  (Elements next to a half in a rarely entered branch, which held
// them in scratch memory: 30000 x 4096 float32 262 us, 99 like this.)
template <int ET>
__device__ __forceinline__ u32x2 quant_eight(const Eight<ET>& x, const Scaling& s) {
  constexpr float kMagic = 12582912.f;
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = x.get(e) * s.up, m = 127.f * v;
    if constexpr (ET == NS_FP32) {
      const float rest = fmaf(127.f, v, -m), f = fmaf(m, s.rcp, kMagic), r = fmaf(kMagic - f, s.a, m);
      const uint32_t u = __float_as_uint(f), neg = __float_as_uint(r) & 0x80000000u;
      const float over = fmaf(-0.5f, s.a, fabsf(r)) + __uint_as_float(__float_as_uint(rest) ^ neg);
      b[e] = u + (over >= __uint_as_float(~u & 1u) ? ((int32_t)neg >> 31) | 1 : 0);
    } else {
      const float q = m * s.rcp;
      b[e] = __float_as_uint(fmaf(fmaf(-q, s.a, m), s.rcp, q) + kMagic);
    }
  }
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
    r[h] = s.ok ? lo | hi : 0u;
  }
  return r;
}

// The row's scale from its maximum's float32 bits.
__device__ __forceinline__ float scale_of(uint32_t m) {
  return m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(m) / 127.f;
}

// Maximum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);    // quad_perm 1 0 3 2
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);             // quad_perm 2 3 0 1
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true);            // row_half_mirror
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true);            // row_mirror
  return o > v ? o : v;
}

constexpr int kQuantThreads = 256;

// T lanes (16, a wave or the block) take a row, G groups of eight elements each.
template <int ET, int T, int G>
__global__ __launch_bounds__(kQuantThreads) void k_quant_rows(const void* __restrict__ x, int64_t ld, int R, int d,
                                                              int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t sh[kQuantThreads / NS_WAVE];
  const int tid = threadIdx.x, t = tid & (T - 1);
  const int64_t r = (int64_t)blockIdx.x * (kQuantThreads / T) + tid / T;
  if (r >= R) return;                              // whole rows
  const int pitch = pitch_of(d);
  const char* row = (const char*)x + (size_t)r * (size_t)ld * (ET == NS_FP32 ? 4 : 2);
  int8_t* out = q + (size_t)r * (size_t)pitch;
  // a load of all lanes covers one run of the row: float32 takes two runs a group
  const auto first = [&](int g) { return ET == NS_FP32 ? (t + 2 * g * T) * 4 : (t + g * T) * 8; };
  const auto put = [&](int g, u32x2 b) {
    const int i = first(g);
    if (ET == NS_FP32) {
      if (i < pitch) *(uint32_t*)(out + i) = b.x;
      if (i + T * 4 < pitch) *(uint32_t*)(out + i + T * 4) = b.y;
    } else if (i < pitch) {
      *(u32x2*)(out + i) = b;
    }
  };
  const int tail = d & ~(ET == NS_FP32 ? 3 : 7);
  const u32x4 rest = Eight<ET>::rest_of(row, tail, d);
  Eight<ET> v[G];
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) v[g].load(row, first(g), T * 4, tail, rest);
  NS_ISSUE_FENCE();
#pragma unroll
  for (int g = 0; g < G; ++g) m = v[g].top(m);
  float top;
  if (ET == NS_FP32) top = __uint_as_float(m);
  else {
    const uint32_t lo = m & 0xFFFFu, hi = m >> 16, b = lo > hi ? lo : hi;
    top = ET == NS_BF16 ? ns::bf16_lo(b) : ns::fp16_lo(b);
  }
  m = __float_as_uint(top);                        // float32 bits order the same way
  if (T == 16) {
    m = row16_max_u32(m);
  } else {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) {
      const uint32_t o = __shfl_xor(m, s, NS_WAVE);
      m = o > m ? o : m;
    }
  }
  if (T > NS_WAVE) {
    if ((tid & 63) == 0) sh[tid / NS_WAVE] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / NS_WAVE; ++w) m = sh[w] > m ? sh[w] : m;
  }
  const Scaling how(m);
#pragma unroll
  for (int g = 0; g < G; ++g) put(g, quant_eight<ET>(v[g], how));
  if (t == 0) scale[r] = scale_of(m);
}

template <int ET>
int quant_rows_of(const void* x, int64_t ld, int R, int d, int8_t* q, float* scale, hipStream_t stream) {
  const int groups = pitch_of(d) / 8;
  // 16 lanes take a row of up to 512 elements (120811 x 87 bf16 in 14 us, 43 with
  // a wave a row; 50000 x 500 16 against 23; 30000 x 1024 20 against 17), a wave
  // one that it can hold if the rows fill the chip without a block each.
  const bool part = groups <= 64, wave = groups <= 8 * NS_WAVE && R >= 1024;
  const int T = part ? 16 : (wave ? NS_WAVE : kQuantThreads), g = (groups + T - 1) / T;
  const dim3 grid((unsigned)((R + kQuantThreads / T - 1) / (kQuantThreads / T))), block(kQuantThreads);
#define NS_LAUNCH_QUANT(TT, G) \
  hipLaunchKernelGGL((k_quant_rows<ET, TT, G>), grid, block, 0, stream, x, ld, R, d, q, scale)
  if (part) {
    if (g <= 1) NS_LAUNCH_QUANT(16, 1);
    else if (g <= 2) NS_LAUNCH_QUANT(16, 2);
    else NS_LAUNCH_QUANT(16, 4);
  } else if (wave) {                               // more than 64 groups: two a lane at least
    if (g <= 2) NS_LAUNCH_QUANT(NS_WAVE, 2);
    else if (g <= 4) NS_LAUNCH_QUANT(NS_WAVE, 4);
    else NS_LAUNCH_QUANT(NS_WAVE, 8);
  } else {
    if (g <= 1) NS_LAUNCH_QUANT(kQuantThreads, 1);
    else if (g <= 2) NS_LAUNCH_QUANT(kQuantThreads, 2);
    else if (g <= 4) NS_LAUNCH_QUANT(kQuantThreads, 4);
    else NS_LAUNCH_QUANT(kQuantThreads, 8);
  }
#undef NS_LAUNCH_QUANT
  return ns_launch_status();
}

int quant_rows(const void* x, int64_t ld, int R, int d, int dtype, int8_t* q, float* scale, hipStream_t stream) {
  if (dtype == NS_BF16) return quant_rows_of<NS_BF16>(x, ld, R, d, q, scale, stream);
  if (dtype == NS_FP16) return quant_rows_of<NS_FP16>(x, ld, R, d, q, scale, stream);
  return quant_rows_of<NS_FP32>(x, ld, R, d, q, scale, stream);
}

// ---------------------------------------------------------------------------
// Integer product
// ---------------------------------------------------------------------------
// Scaled value of an exact integer sum.
__device__ __forceinline__ float scaled(int acc, float s) { return (float)acc * s; }

// A float32 value as it is: without this the compiler forms mixed-precision
// multiplies that round a product to fp16 at once.
__device__ __forceinline__ float as_float32(float v) {
  asm("" : "+v"(v));
  return v;
}

template <int OT>
__device__ __forceinline__ void store_out(void* out, size_t i, float v) {
  if (OT == NS_FP32) ((float*)out)[i] = v;
  else if (OT == NS_BF16) ((__bf16*)out)[i] = (__bf16)v;
  else ((_Float16*)out)[i] = (_Float16)as_float32(v);
}

struct Product {
  const int8_t* x;          // [B][M][pitch]
  const float* xs;          // [B][M]
  const int8_t* w;          // [rows][pitch]
  const float* ws;          // [rows]
  const int32_t* ids;       // [B][N] row of column j, or NULL: j
  const int32_t* n_dev;     // [B] live columns, or NULL: N
  int M, N, V, pitch;
  void* out;                // [B][M][N], elements of a token `sm` apart for m, `sn` for n
  int64_t sm, sn;
};

constexpr int kStageK = 128;                       // bytes of a row in a stage

// 16 bytes a lane from a buffer straight into LDS at byte `lds` (the same
// for the wave) + 16 * lane.  The compiler does not count these loads: the
// waits below do.  m0 holds the LDS address.  The compiler does not see a
// memory instruction here either, so the asm keeps the distances itself: the
// move and the no-ops are the five wait states from a vector instruction that
// wrote an SGPR (v_readlane, as for a spilled one) to a memory instruction that
// reads it, and more than the one from the move to the load.  m0 is a register
// that the compiler reserves and writes before each use of its own, so it warns
// of the clobber, which tells it that the value is gone.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
               : "memory", "m0");
}

// The same for bytes that are read once: the caches need not keep them.
__device__ __forceinline__ void load_to_lds_once(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
               : "memory", "m0");
}

// The same for four bytes a lane.
__device__ __forceinline__ void load_word_to_lds(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
               : "memory", "m0");
}

#pragma clang diagnostic pop

__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, 0x00027000u};
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

template <int OT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if (OT == NS_BF16) {
    const __bf16 x = (__bf16)a, y = (__bf16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
  }
  const _Float16 x = (_Float16)as_float32(a), y = (_Float16)as_float32(b);
  return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
}

// Eight consecutive outputs, n of them inside the row.
template <int OT>
__device__ __forceinline__ void store_eight(void* out, size_t i, const float (&v)[8], int n) {
  if (n >= 8) {
    if (OT == NS_FP32) {
      u32x4_any* d = (u32x4_any*)((float*)out + i);
      d[0] = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      d[1] = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
      *(u32x4_any*)((uint16_t*)out + i) = u32x4{narrow2<OT>(v[0], v[1]), narrow2<OT>(v[2], v[3]),
                                                narrow2<OT>(v[4], v[5]), narrow2<OT>(v[6], v[7])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) store_out<OT>(out, i + e, v[e]);
  }
}

// ---------------------------------------------------------------------------
// The product for up to 128 token rows: bound by the bytes of the channel rows,
// each read once.
//
// One block of eight waves a CU takes an even share of the 16-row channel
// units and runs through it in passes of 8 RT units, RT a wave, in stages of
// 128 bytes a row.  A ring of stages in LDS is filled by direct
// global-to-LDS loads, R - 1 stages ahead (72 to 132 KB a CU, 48 to 96 KB of
// them channel rows), across the ends of passes; channel rows are private to
// their wave, token rows shared by the block, so one barrier a stage orders the
// ring.  Waits count the loads
// that may still be out; outputs leave by buffer stores, which out-of-range
// lanes take part in without effect, so the stores behind a pass are as many
// for every pass and the waits can allow for them.
//
// Block b begins every row at stage 5 b mod S and goes round (the sum is
// exact in any order): blocks that walked along their rows in step would read
// addresses alike in their low bits, a few memory channels' worth.  8 x 128256
// x 4096: 98.9 -> 79.0 us (6.6 TB/s).
//
// The token rows are operand A and the channel rows operand B, so 16 lanes
// hold 16 consecutive outputs of a token.  Place c of row r in LDS holds
// 16-byte chunk c ^ (r % 8): no bank is met twice.
// More than 32 tokens take RT = 2: a stage's token rows, which all eight waves
// read from LDS, then serve twice the channel rows (60 x 151936 x 3584: 110
// -> 103 us, 5.5 TB/s with the outputs; 8 x 128256 x 4096 79 -> 81 us).
// Without the output stores it takes 89 us; stores of two outputs a lane took
// as long as these.
// ---------------------------------------------------------------------------
constexpr int kStreamWaves = 8;

// With IDS the channel rows are those that ids names (n_dev of them), the
// block's share of ids waiting in LDS, and blockIdx.y is the sequence.
constexpr int kStreamIds = 4096;                     // ids of a block, at most

template <int OT, int NMT, int ROWS, int R, bool IDS>
__global__ __launch_bounds__(kStreamWaves* NS_WAVE, 2) void k_product_stream(Product p) {
  constexpr int RT = ROWS > 16 ? ROWS / 16 : 1, PROWS = kStreamWaves * ROWS, LR = ROWS / 8;
  constexpr int XOFF = PROWS * kStageK, SOFF = XOFF + NMT * 16 * kStageK;
  constexpr int STAGE = SOFF + kStreamWaves * 256;   // channel rows, token rows, channel scales
  constexpr int XL = NMT % 4 == 0 ? NMT / 4 : NMT, LW = LR + XL;   // loads of a wave and stage
  // stores behind a pass that the waits allow for (vmcnt counts to 63)
  constexpr int STORES = RT * NMT * 4 < 63 - (R - 2) * LW ? RT * NMT * 4 : 63 - (R - 2) * LW;
  static_assert((R - 2) * LW + STORES < 64, "vmcnt range");
  __shared__ __attribute__((aligned(16))) char lds[R * STAGE];
  __shared__ int s_id[IDS ? kStreamIds : 1];
  int live = p.N;
  if (IDS) {
    const size_t seq = blockIdx.y;
    if (p.n_dev) live = p.n_dev[seq] < 0 ? 0 : (p.n_dev[seq] < p.N ? p.n_dev[seq] : p.N);
    p.x += seq * p.M * p.pitch;
    p.xs += seq * p.M;
    if (p.ids) p.ids += seq * p.N;
    p.out = (char*)p.out + seq * p.M * (size_t)p.sm * (OT == NS_FP32 ? 4 : 2);
  }
  const int units = (live + ROWS - 1) / ROWS, per_block = (units + (int)gridDim.x - 1) / (int)gridDim.x;
  const int u0 = (int)blockIdx.x * per_block, u1 = u0 + per_block < units ? u0 + per_block : units;
  const int passes = (u1 - u0 + kStreamWaves - 1) / kStreamWaves;
  if (passes <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
  const int S = p.pitch / kStageK;
  const uint32_t base = lds_offset(lds);
  const int n0 = u0 * ROWS;                            // the block's first channel row
  const int last = (u1 * ROWS < live ? u1 * ROWS : live) - 1 - n0;
  const u32x4 rw = IDS ? buffer_of(p.w, (uint32_t)p.V * p.pitch)
                       : buffer_of(p.w + (size_t)n0 * p.pitch, (uint32_t)(last + 1) * p.pitch);
  const u32x4 rx = buffer_of(p.x, (uint32_t)(p.M * p.pitch));
  const u32x4 rs = IDS ? buffer_of(p.ws, (uint32_t)p.V * 4) : buffer_of(p.ws + n0, (uint32_t)(last + 1) * 4);
  float xs[NMT][4];
#pragma unroll
  for (int u = 0; u < NMT; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = u * 16 + g * 4 + r;
      xs[u][r] = p.xs[m < p.M ? m : p.M - 1];
    }
  if (IDS) {                                         // a hole reads row 0; nobody reads its output
    for (int r = tid; r <= last; r += kStreamWaves * NS_WAVE) {
      const int id = p.ids ? p.ids[n0 + r] : n0 + r;
      s_id[r] = id < 0 || id >= p.V ? 0 : id;
    }
    __syncthreads();
  }
  // token rows past the end read the last one and are not stored
  uint32_t xo[XL];
  if (NMT % 4 == 0) {
#pragma unroll
    for (int v = 0; v < XL; ++v) {
      const int r = (v * 8 + w) * 8 + (lane >> 3);
      xo[v] = (uint32_t)((r < p.M ? r : p.M - 1) * p.pitch + ((lane & 7) ^ (lane >> 3)) * 16);
    }
  } else {
#pragma unroll
    for (int v = 0; v < NMT; ++v) {                  // two rows a load, a word a lane
      const int r = v * 16 + w * 2 + (lane >> 5), q = lane & 31;
      xo[v] = (uint32_t)((r < p.M ? r : p.M - 1) * p.pitch + (((q >> 2) ^ (r & 7)) * 4 + (q & 3)) * 4);
    }
  }
  // The stream of loads: the lk-th stage of pass lp comes next, bytes ks of the rows, into place lb.
  int lp = 0, lk = 0, lb = 0, ks = (int)(blockIdx.x * 5u) % S * kStageK;
  uint32_t wo[LR], so;                           // of the pass
  const auto aim = [&]() {
    const int r0 = (lp * kStreamWaves + w) * ROWS;
    const auto row = [&](int r) {
      r = r < last ? r : last;
      return (uint32_t)(IDS ? s_id[r] : r);
    };
#pragma unroll
    for (int v = 0; v < LR; ++v)
      wo[v] = __umul24(row(r0 + v * 8 + (lane >> 3)), p.pitch) + ((lane & 7) ^ (lane >> 3)) * 16;
    so = row(r0 + (lane & (ROWS - 1))) * 4;
  };
  const auto issue = [&]() {
    const uint32_t to = base + lb * STAGE;
#pragma unroll
    for (int v = 0; v < LR; ++v) load_to_lds_once(rw, wo[v], ks, to + (w * LR + v) * 1024);
    if (NMT % 4 == 0) {
#pragma unroll
      for (int v = 0; v < XL; ++v) load_to_lds(rx, xo[v], ks, to + XOFF + (v * 8 + w) * 1024);
    } else {
#pragma unroll
      for (int v = 0; v < NMT; ++v) load_word_to_lds(rx, xo[v], ks, to + XOFF + (v * 8 + w) * 256);
    }
    if (lk == 0) load_word_to_lds(rs, so, 0, to + SOFF + w * 256);
    lb = lb + 1 == R ? 0 : lb + 1;
    ks = ks + kStageK == p.pitch ? 0 : ks + kStageK;
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
  i32x4 acc[RT][NMT] = {};
  // the scales are here before the loads are counted
#pragma unroll
  for (int u = 0; u < NMT; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) asm volatile("" : "+v"(xs[u][r]));
#pragma unroll
  for (int v = 0; v < R - 1; ++v) issue();
  const int place0 = (g ^ (i & 7)) * 16, place1 = ((4 + g) ^ (i & 7)) * 16;
  const int ir = ROWS < 16 ? i & (ROWS - 1) : i;     // with 8 rows the operand's upper half repeats the lower
  const char* lw = lds + (w * ROWS + ir) * kStageK;
  const char* lx = lds + XOFF + i * kStageK;
  int b = 0, since = R;                              // stages since the last stores
  float ws[RT] = {};
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
      if (s == 0) {
#pragma unroll
        for (int t = 0; t < RT; ++t) ws[t] = *(const float*)(lds + b * STAGE + SOFF + w * 256 + (t * 16 + ir) * 4);
      }
      i32x4 f[RT][2];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        f[t][0] = *(const i32x4*)(at + t * 16 * kStageK + place0);
        f[t][1] = *(const i32x4*)(at + t * 16 * kStageK + place1);
      }
#pragma unroll
      for (int u = 0; u < NMT; ++u) {
        const i32x4 x0 = *(const i32x4*)(xt + u * 16 * kStageK + place0);
        const i32x4 x1 = *(const i32x4*)(xt + u * 16 * kStageK + place1);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x0, f[t][0], acc[t][u], 0, 0, 0);
          acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x1, f[t][1], acc[t][u], 0, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);             // no read moves behind the wait
      __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0): this wave has read the stage
      b = b + 1 == R ? 0 : b + 1;
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int j = (pass * kStreamWaves + w) * ROWS + t * 16 + i;
#pragma unroll
      for (int u = 0; u < NMT; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int m = u * 16 + g * 4 + r;
          const float v = scaled(acc[t][u][r], xs[u][r] * ws[t]);
          const uint32_t at =
              m < p.M && j <= last && (ROWS >= 16 || i < ROWS) ? (uint32_t)(((size_t)m * (size_t)p.sm + (size_t)(n0 + j) * (size_t)p.sn) * ESZ) : 0x80000000u;
          if (OT == NS_FP32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), ro, at, 0, 0);
          else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)narrow2<OT>(v, 0.f), ro, at, 0, 0);
          acc[t][u][r] = 0;
        }
    }
    since = 0;
  }
  wait_loads<0>();                                   // the stream's last loads end before their LDS is given back
}

// ---------------------------------------------------------------------------
// The product for more than 64 token rows: compute-bound, tiles in LDS.
//
// A block of eight waves owns 256 channel rows and TB * 64 token rows of the
// output; a wave owns 128 channel rows (eight operands of 16) and TB * 16
// token rows (TB operands), 8 TB accumulator tiles in registers.  The sum runs
// in stages of 128 bytes a row, two in LDS (68 KB each with TB = 4), three with
// TB = 1, whose short stages end before a load does (256 x 16384 x 4096, a tile
// a CU: 29.5 -> 25.3 us), filled by direct global-to-LDS loads.  While one half
// of a stage (64 bytes a row) is multiplied, the next half is read into a second
// set of registers; once a wave holds a stage's second half and the next stage
// has landed, one block barrier frees the stage's place for the stage after next.
//
// Blocks stay: each takes one tile after the other, and the stages of all its
// tiles (with the tiles' scales) are one stream of loads, so the next tile's
// first stages arrive while the last ones of this tile are multiplied and its
// outputs are stored.  Tiles go to the blocks of one XCD from one contiguous
// run, in groups of four channel tiles by all token tiles, so that its 32 CUs
// share rows in its L2.
//
// Lane i of channel operand t is channel row 8 i + t, so the eight
// accumulators of a lane are eight consecutive outputs and a store of 16
// lanes covers 128 of them, without a detour through LDS.
//
// 4096 x 128256 x 4096 takes 1655 to 1730 us (2.5 to 2.6 POP/s): the matrix units
// are busy for 74 % of the cycles, and the clock gives way under the load.
// Products of 32 x 32 x 32 (1841 us) and four stages of 64 bytes (1911) were
// slower.
//
// Place c of row r in LDS holds 16-byte chunk c ^ (r / 8 % 8) of channel rows and
// c ^ (r % 8) of token rows, and eight channel rows stand 128 bytes from the next
// eight, so that lanes i and i + 1 read from different halves of the 64 banks: no
// bank is met twice (without that 128 bytes a fifth of the cycles were conflicts;
// 1024 x 128256 x 4096 482 -> 467 us).
// ---------------------------------------------------------------------------
constexpr int kTileN = 256;                        // channel rows of a block
constexpr int kTileThreads = 512;
constexpr int tile_stages(int tb) { return tb == 1 ? 3 : 2; }   // in LDS
constexpr int kEightRows = 9 * kStageK;            // eight channel rows in LDS and 128 bytes between them and the next

template <int OT, int TB>
__global__ __launch_bounds__(kTileThreads, 2) void k_product_tiled(Product p, int tiles_m, int tiles_n) {
  constexpr int TM = TB * 64;                      // token rows of a block
  constexpr int XOFF = kTileN / 8 * kEightRows, STAGE = XOFF + TM * kStageK;
  constexpr int LA = kTileN / 64, LB = TM / 64;    // loads of a wave and stage: 8 rows each
  constexpr int STORES = TB * 4 * (OT == NS_FP32 ? 2 : 1);   // of a wave and whole tile
  constexpr int R = tile_stages(TB), AHEAD = (R - 2) * (LA + LB);   // loads that may be out when a stage must be here
  static_assert(AHEAD + STORES < 64, "vmcnt range");
  // scales of the tile that is multiplied and, with one stage a tile, of R more
  __shared__ __attribute__((aligned(16))) char lds[R * STAGE + (R + 1) * 2048];
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
  const int S = p.pitch / kStageK;
  const uint32_t base = lds_offset(lds);

  // The stream of loads: stage `lk` of tile `lt` comes next.
  int lt = tile, lk = 0, to_scales = 0;
  u32x4 ra, rb, rs;
  int last_a, last_b, last_s;                      // rows past the end read the last one and are not stored
  const auto aim = [&]() {
    int m0, n0;
    origin(lt, m0, n0);
    last_a = p.N - 1 - n0;
    last_b = p.M - 1 - m0;
    last_s = w < 4 ? last_a : last_b;
    ra = buffer_of(p.w + (size_t)n0 * p.pitch, (uint32_t)(kTileN * p.pitch));
    rb = buffer_of(p.x + (size_t)m0 * p.pitch, (uint32_t)(TM * p.pitch));
    // scales: waves 0 to 3 the channels', waves 4 to 7 the tokens', 64 each
    rs = buffer_of(w < 4 ? p.ws + n0 : p.xs + m0, 1024);
  };
  // Load u of the next stage's LA + LB, into buffer buf.
  const auto load = [&](int u, int buf) {
    int l = lane;                                  // opaque: the few values below are computed anew each
    asm volatile("" : "+v"(l));                    // time instead of being held in registers all along
    const int v = u < LA ? u : u - LA, r = (v * 8 + w) * 8 + (l >> 3), last = u < LA ? last_a : last_b;
    const int chunk = (l & 7) ^ (u < LA ? w : l >> 3);
    load_to_lds(u < LA ? ra : rb, __umul24(r < last ? r : last, p.pitch) + chunk * 16, lk * kStageK,
                base + buf * STAGE + (u < LA ? (v * 8 + w) * kEightRows : XOFF + (v * 8 + w) * 8 * kStageK));
  };
  // Behind a stage's loads: the tile's scales with its first stage, then on to the next stage.
  const auto advance = [&]() {
    if (lk == 0) {
      int l = lane;
      asm volatile("" : "+v"(l));
      const int q = (w & 3) * 64 + l;
      load_word_to_lds(rs, (uint32_t)(q < last_s ? q : last_s) * 4, 0, base + R * STAGE + to_scales * 2048 + w * 256);
      to_scales = to_scales == R ? 0 : to_scales + 1;
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
  i32x4 acc[8][TB] = {};
  // The channel operands of the half that is multiplied, 6 and 7 apart: the
  // next half's replace 0 to 5 as they fall free, and 6 and 7 alternate, so
  // that no read is still to come behind the half's last products.
  i32x4 fa[6], fe[2][2], fb[2][TB];
  // operand t: channel rows wr * 128 + 8 i + t; operand u: token rows (wc * TB + u) * 16 + i
  const char* la = lds + (wr * 16 + i) * kEightRows;
  const char* lb = lds + XOFF + (wc * TB * 16 + i) * kStageK;
  const int place0 = (g ^ (i & 7)) * 16, place1 = ((4 + g) ^ (i & 7)) * 16;
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
#pragma unroll
  for (int u = 0; u < TB; ++u) fb[0][u] = *(const i32x4*)(lb + place0 + u * 16 * kStageK);
#pragma unroll
  for (int t = 0; t < 6; ++t) fa[t] = *(const i32x4*)(la + place0 + t * kStageK);
  fe[0][0] = *(const i32x4*)(la + place0 + 6 * kStageK);
  fe[0][1] = *(const i32x4*)(la + place0 + 7 * kStageK);
  // Multiplies the half in registers (fe, fb of f) and reads the next from
  // `at`.  With `more`, the next stage's loads go out between the products,
  // one for each operand: eight waves that issue theirs all at once wait for
  // the load unit (64 KB at 64 bytes a cycle) with their products behind them.
  const auto step = [&](int f, int at, bool more, int buf) {
#pragma unroll
    for (int u = 0; u < TB; ++u) fb[1 - f][u] = *(const i32x4*)(lb + at + u * 16 * kStageK);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (more && t < LA + LB) load(t, buf);
      const i32x4 a = t < 6 ? fa[t % 6] : fe[f][t & 1];
#pragma unroll
      for (int u = 0; u < TB; ++u) acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[f][u], a, acc[t][u], 0, 0, 0);
      if (t < 6) fa[t % 6] = *(const i32x4*)(la + at + t * kStageK);
      if (t == 3 || t == 4) fe[1 - f][t - 3] = *(const i32x4*)(la + at + (t + 3) * kStageK);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int b = 0, scales = 0;
  bool stored = false;                             // the tile before was whole: STORES stores are behind the loads
  for (; tile < end; tile += slots) {
    for (int s = 0; s < S; ++s) {
      step(0, b * STAGE + place1, false, 0);
      __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0): this wave has read the stage
      if (s == 0 && stored) wait_loads<AHEAD + STORES>();
      else wait_loads<AHEAD>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      const int next = b + 1 == R ? 0 : b + 1;
      step(1, next * STAGE + place0, true, b);
      advance();
      b = next;
    }
    int m0, n0, l = lane;
    asm volatile("" : "+v"(l));                    // as in load
    const int ni = (l & 15) * 8, mg = (l >> 4) * 4;
    origin(tile, m0, n0);
    const float* sw = (const float*)(lds + R * STAGE + scales * 2048) + wr * 128 + ni;
    const float* sx = (const float*)(lds + R * STAGE + scales * 2048) + 256 + wc * TB * 16 + mg;
    scales = scales == R ? 0 : scales + 1;
    float ws[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) ws[e] = sw[e];
    const int n = n0 + wr * 128 + ni;
    stored = m0 + TM <= p.M && n0 + kTileN <= p.N;
#pragma unroll
    for (int u = 0; u < TB; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = m0 + (wc * TB + u) * 16 + mg + r;
        const float xs = sx[u * 16 + r];
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = scaled(acc[e][u][r], xs * ws[e]);
        const size_t at = (size_t)m * (size_t)p.sm + n;
        if (stored) store_eight<OT>(p.out, at, v, 8);
        else if (m < p.M && n < p.N) store_eight<OT>(p.out, at, v, p.N - n);
      }
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int u = 0; u < TB; ++u) acc[t][u] = i32x4{0, 0, 0, 0};
  }
  wait_loads<0>();                                 // the stream's last loads end before their LDS is given back
}

// ---------------------------------------------------------------------------
// The product for few channel rows: bound by latency.  A block of eight waves
// owns 16 channel rows and up to 64 token rows (blockIdx.z of them); each wave
// takes an eighth of the row's bytes, asks for all of its operands at once
// and multiplies; the eight sums are joined in LDS.  One block pulls 64 KB of
// a 4096-byte row set in about a microsecond, and 63 blocks of a thousand
// rows end together.
// ---------------------------------------------------------------------------
template <int OT, int NMT>
__global__ __launch_bounds__(512) void k_product_few(Product p) {
  constexpr int BATCH = NMT == 1 ? 8 : 4;            // operands of a row in flight
  __shared__ i32x4 sh[8][NMT][NS_WAVE];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, i = lane & 15, g = lane >> 4;
  const int m0 = (int)blockIdx.z * NMT * 16;         // tokens in groups
  p.x += (size_t)m0 * p.pitch;
  p.xs += m0;
  p.out = (char*)p.out + (size_t)m0 * (size_t)p.sm * (OT == NS_FP32 ? 4 : 2);
  const size_t seq = blockIdx.y;
  const int M = p.M - m0;                            // tokens from here on
  const int j0 = (int)blockIdx.x * 16, j = j0 + i < p.N ? j0 + i : p.N - 1;
  // the count, the ids and the scales are asked for together; an id behind
  // the count or a hole reads some row, and nobody reads its output
  int n = p.n_dev ? p.n_dev[seq] : p.N;
  int id = p.ids ? p.ids[seq * p.N + j] : j;
  float xs[NMT][4];
#pragma unroll
  for (int u = 0; u < NMT; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = u * 16 + g * 4 + r;
      xs[u][r] = p.xs[seq * p.M + (m < M ? m : M - 1)];
    }
  NS_ISSUE_FENCE();
  n = n < p.N ? n : p.N;
  if (j0 >= n) return;
  id = id < 0 || id >= p.V ? 0 : id;
  const float ws = p.ws[id];
  const int steps = p.pitch / 64, per = (steps + 7) / 8;
  const int k0 = w * per, k1 = k0 + per < steps ? k0 + per : steps;
  const int8_t* wr = p.w + (size_t)id * p.pitch + g * 16;
  const int8_t* xr[NMT];
#pragma unroll
  for (int u = 0; u < NMT; ++u) {
    const int m = u * 16 + i < M ? u * 16 + i : M - 1;
    xr[u] = p.x + (seq * p.M + m) * p.pitch + g * 16;
  }
  i32x4 acc[NMT] = {};
  for (int k = k0; k < k1; k += BATCH) {
    i32x4 a[BATCH], b[BATCH][NMT];
#pragma unroll
    for (int q = 0; q < BATCH; ++q) {
      const int at = (k + q < k1 ? k + q : k0) * 64;
      a[q] = *(const i32x4*)(wr + at);
#pragma unroll
      for (int u = 0; u < NMT; ++u) b[q][u] = *(const i32x4*)(xr[u] + at);
    }
    NS_ISSUE_FENCE();
#pragma unroll
    for (int q = 0; q < BATCH; ++q)
      if (k + q < k1) {                              // uniform over the wave
#pragma unroll
        for (int u = 0; u < NMT; ++u) acc[u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[q][u], a[q], acc[u], 0, 0, 0);
      }
  }
#pragma unroll
  for (int u = 0; u < NMT; ++u) sh[w][u][lane] = acc[u];
  __syncthreads();
  // wave u joins token operand u; lane (i, g) holds tokens 4 g .. 4 g + 3 of channel i
#pragma unroll
  for (int u = 0; u < NMT; ++u) {
    if (u != w) continue;
    i32x4 s = sh[0][u][lane];
#pragma unroll
    for (int q = 1; q < 8; ++q) s += sh[q][u][lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = u * 16 + g * 4 + r;
      if (m < M && j0 + i < n)
        store_out<OT>(p.out, (seq * p.M + m) * (size_t)p.sm + (size_t)(j0 + i) * (size_t)p.sn, scaled(s[r], xs[u][r] * ws));
    }
  }
}

// ---------------------------------------------------------------------------
// The head over few rows with the quantisation of its hidden rows in the same
// launch, for up to 16 of them, 32 KB of 8-bit hidden rows and d % 8 = 0: every
// block quantises them all into LDS (U groups of eight elements a thread) while
// its channel rows are on their way.  A launch less: M = 8, d = 4096, 1000 rows
// 12.6 -> 12.0 us, M = 1 11.8 -> 8.8, 19 sequences of 46 rows, M = 8, d = 320,
// 12.5 -> 9.8.  Bound by latency and by that quantisation: at 1000 rows and d =
// 4096 the kernel takes 8.5 us with M = 8, 5.0 with M = 1, k_product_few over rows
// quantised before 5.7 and 4.7.
// ---------------------------------------------------------------------------
constexpr int kFusedBytes = 32768;                 // M * pitch, at most
constexpr int kFusedPad = 16;                      // between token rows in LDS: no bank is met twice

template <int ET, int U>
__global__ __launch_bounds__(512) void k_head_few(Product p, const void* __restrict__ h, int d) {
  constexpr int BATCH = 8;
  __shared__ __attribute__((aligned(16))) char xq[kFusedBytes + 16 * kFusedPad];
  __shared__ i32x4 sh[8][NS_WAVE];
  __shared__ uint32_t s_top[16];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, i = lane & 15, g = lane >> 4;
  const size_t seq = blockIdx.y;
  const int j0 = (int)blockIdx.x * 16, j = j0 + i < p.N ? j0 + i : p.N - 1;
  int n = p.n_dev ? p.n_dev[seq] : p.N;
  int id = p.ids ? p.ids[seq * p.N + j] : j;
  // Hidden rows in chunks of 128 elements, 16 lanes each, lane c % 16 eight of
  // them; c / per_row by a product, exact for c * per_row < 2^16.
  const int per_row = p.pitch / 128, chunks = p.M * per_row, magic = 65536 / per_row + 1;
  const char* hb = (const char*)h + seq * p.M * (size_t)d * (ET == NS_FP32 ? 4 : 2);
  Eight<ET> v[U];
  int tok[U], at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (tid >> 4) + u * 32;
    tok[u] = c < chunks ? c * magic >> 16 : -1;
    at[u] = (c - tok[u] * per_row) * 128 + (tid & 15) * 8;
    // a group past the last row reads the first, and nobody reads it
    v[u].load(hb + (size_t)(tok[u] < 0 ? 0 : tok[u]) * d * (ET == NS_FP32 ? 4 : 2), at[u], 4, d, u32x4{0, 0, 0, 0});
  }
  if (tid < 16) s_top[tid] = 0;
  NS_ISSUE_FENCE();
  n = n < p.N ? n : p.N;
  if (j0 >= n) return;
  id = id < 0 || id >= p.V ? 0 : id;
  const float ws = p.ws[id];
  const int steps = p.pitch / 64, per = (steps + 7) / 8;
  const int k0 = w * per, k1 = k0 + per < steps ? k0 + per : steps;
  const int8_t* wr = p.w + (size_t)id * p.pitch + g * 16;
  i32x4 a[BATCH];
  const auto rows = [&](int k) {
#pragma unroll
    for (int q = 0; q < BATCH; ++q) a[q] = *(const i32x4*)(wr + (k + q < k1 ? k + q : 0) * 64);
  };
  rows(k0);
  NS_ISSUE_FENCE();
  const auto sync = [&]() {                          // LDS only: the loads stay out
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  sync();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (tok[u] < 0) continue;                        // whole rows of 16 lanes
    const uint32_t t = v[u].top(0);
    float top;
    if (ET == NS_FP32) top = __uint_as_float(t);
    else {
      const uint32_t lo = t & 0xFFFFu, hi = t >> 16, b = lo > hi ? lo : hi;
      top = ET == NS_BF16 ? ns::bf16_lo(b) : ns::fp16_lo(b);
    }
    const uint32_t most = row16_max_u32(__float_as_uint(top));
    if ((tid & 15) == 0) atomicMax(&s_top[tok[u]], most);
  }
  sync();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (tok[u] < 0) continue;
    const u32x2 q = quant_eight<ET>(v[u], Scaling(s_top[tok[u]]));
    *(u32x2*)(xq + tok[u] * (p.pitch + kFusedPad) + at[u]) = q;
  }
  sync();
  const char* xr = xq + (i < p.M ? i : 0) * (p.pitch + kFusedPad) + g * 16;
  i32x4 acc = {};
  for (int k = k0; k < k1; k += BATCH) {
    if (k > k0) rows(k);
#pragma unroll
    for (int q = 0; q < BATCH; ++q)
      if (k + q < k1) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*(const i32x4*)(xr + (k + q) * 64), a[q], acc, 0, 0, 0);
  }
  sh[w][lane] = acc;
  __syncthreads();
  if (w != 0) return;
  i32x4 s = sh[0][lane];
#pragma unroll
  for (int q = 1; q < 8; ++q) s += sh[q][lane];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int m = g * 4 + r;
    if (m >= p.M || j0 + i >= n) continue;
    const float xs = scale_of(s_top[m]);
    store_out<NS_FP32>(p.out, (seq * p.M + m) * (size_t)p.sm + (size_t)(j0 + i) * (size_t)p.sn, scaled(s[r], xs * ws));
  }
}

template <int ET>
void launch_head_few(const Product& p, int B, const void* h, int d, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)B), block(512);
  if (p.M * p.pitch <= kFusedBytes / 4) hipLaunchKernelGGL((k_head_few<ET, 2>), grid, block, 0, stream, p, h, d);
  else hipLaunchKernelGGL((k_head_few<ET, 8>), grid, block, 0, stream, p, h, d);
}

template <int OT, int TB>
void launch_tiled(const Product& p, hipStream_t stream) {
  const int tm = (p.M + TB * 64 - 1) / (TB * 64), tn = (p.N + kTileN - 1) / kTileN;
  // one block a CU, eight XCDs of 32 CUs
  const unsigned per = ((unsigned)tm * (unsigned)tn + 7) / 8;
  hipLaunchKernelGGL((k_product_tiled<OT, TB>), dim3((per < 32 ? per : 32) * 8), dim3(kTileThreads), 0, stream, p, tm,
                     tn);
}

template <int OT, int NMT, int ROWS, int R>
void launch_stream(const Product& p, hipStream_t stream) {
  const int units = (p.N + ROWS - 1) / ROWS, per = (units + 255) / 256;
  hipLaunchKernelGGL((k_product_stream<OT, NMT, ROWS, R, false>), dim3((unsigned)((units + per - 1) / per)),
                     dim3(kStreamWaves * NS_WAVE), 0, stream, p);
}

template <int OT, int NMT>
void launch_few(const Product& p, int B, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)B, (unsigned)((p.M + NMT * 16 - 1) / (NMT * 16)));
  hipLaunchKernelGGL((k_product_few<OT, NMT>), grid, dim3(512), 0, stream, p);
}

template <int OT>
void launch_few_of(const Product& p, int B, hipStream_t stream) {
  if (p.M <= 16) launch_few<OT, 1>(p, B, stream);
  else if (p.M <= 32) launch_few<OT, 2>(p, B, stream);
  else if (p.M <= 48) launch_few<OT, 3>(p, B, stream);
  else launch_few<OT, 4>(p, B, stream);
}

// Up to 64 tokens: up to 4096 channels (a 16-row block a CU) the kernel for few
// rows (M = 8, d = 4096: 2048 channels 5.7 us against 10.5 streamed, 4096 6.1
// against 10.7, 10000 13.3 against 11.4); up to 16384 (one pass of eight-row
// units) the stream of those (M = 60, d = 3584: 16000 channels 15.0 us against
// 21.1 with taller units, 30000 28.8 against 23.9); then the taller units.
// Up to 128 tokens over more than 65536 channels the stream still is the faster
// (151936 channels, d = 3584: 65 tokens 128 against 144 us in tiles, 128 138
// against 151; d = 4096: 128 tokens, 128256 channels 109 against 138, 60000 as
// fast, 20000 40 against 32).  With at most 64 channels the
// two sides change places.  More than 64 tokens over few channels also go to
// the kernel for few rows, 64 at a time, up to a block a CU (321 x 184 x 9508
// 25 us against 82 in tiles of 256 tokens; 100 x 2000 x 16384, 250 blocks, 39
// against 98; 128 x 2560 x 4096, 320 blocks, 21.9 against 20.0 in tiles of 64).
// The rest takes tiles of 256, 128 or 64 tokens.  Blocks take one tile each a
// round, and a round takes about 42, 30 and 22 us at d = 4096 (256 x 16384,
// one round each: 43.1, 31.6, 25.3); the sum over the rounds decides (1000 x
// 8000 x 4096, rounds 1, 1 and 2: 48.4, 37.1, 46.9; 3000 x 10000 x 500, rounds
// 2, 4 and 8: 24.8, 26.9, 35.6; 4096 x 128256 x 4096 1665, 2073, 2694).
template <int OT>
void launch_product(Product p, hipStream_t stream) {
  if (p.M > 64 && p.N <= 64) {
    p = Product{p.w, p.ws, p.x, p.xs, nullptr, nullptr, p.N, p.M, p.M, p.pitch, p.out, p.sn, p.sm};
  }
  const uint64_t span = ((uint64_t)(p.M - 1) * (uint64_t)p.sm + (uint64_t)(p.N - 1) * (uint64_t)p.sn + 1) *
                        (OT == NS_FP32 ? 4 : 2);
  const int64_t few = (int64_t)((p.N + 15) / 16) * ((p.M + 63) / 64);   // blocks of the kernel for few rows
  if ((p.M <= 64 && p.N <= 4096) || (p.M > 64 && few <= 256)) {
    launch_few_of<OT>(p, 1, stream);
  } else if (p.M <= 64 && span < 0x7FFFFFFFull) {    // the stream's output offsets have 31 bits
    if (p.N <= 16384) {
      if (p.M <= 16) launch_stream<OT, 1, 8, 7>(p, stream);
      else if (p.M <= 32) launch_stream<OT, 2, 8, 7>(p, stream);
      else if (p.M <= 48) launch_stream<OT, 3, 8, 7>(p, stream);
      else launch_stream<OT, 4, 8, 7>(p, stream);
    } else {
      if (p.M <= 16) launch_stream<OT, 1, 16, 7>(p, stream);
      else if (p.M <= 32) launch_stream<OT, 2, 16, 7>(p, stream);
      else if (p.M <= 48) launch_stream<OT, 3, 32, 3>(p, stream);
      else launch_stream<OT, 4, 32, 3>(p, stream);
    }
  } else if (p.M <= 64) {
    launch_few_of<OT>(p, 1, stream);
  } else if (p.M <= 128 && p.N > 65536 && span < 0x7FFFFFFFull) {
    launch_stream<OT, 8, 32, 3>(p, stream);
  } else {
    const auto time = [&](int tb, int round) {
      const int64_t tiles = (int64_t)((p.N + kTileN - 1) / kTileN) * ((p.M + tb * 64 - 1) / (tb * 64));
      return (tiles + 255) / 256 * round;
    };
    const int64_t t4 = time(4, 21), t2 = time(2, 15), t1 = time(1, 11);
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
  hipLaunchKernelGGL((k_product_stream<NS_FP32, NMT, ROWS, R, true>), dim3((unsigned)gx, (unsigned)B),
                     dim3(kStreamWaves * NS_WAVE), 0, stream, p);
}

// The head's logits, B sequences.  Whole calls, the kernel for few rows
// against the stream of eight-row units: M = 8, 1000 rows 13.4 against 18.2 us;
// M = 64, 4000 rows 23.0 against 26.4, 8000 rows 36.5 against 31.4, 15500 rows
// 54.1 against 33.0; 32 sequences of 1000 of 2048 rows, M = 8, 42.2 against
// 30.3.  Taller units, with fewer barriers, pay once a CU has several passes
// of eight-row ones (M = 8, 100000 rows 81.4 against 83.7 us; 15500 rows, M =
// 64, 39.3 against 33.0).  The stream's 32-bit row addresses reach 4 GB.
bool few_rows(int B, int n_max, int V, int d) {
  return (int64_t)B * n_max < 8192 || (uint64_t)V * (uint64_t)pitch_of(d) > 0xFFFFFFFFull;
}

void launch_head(const Product& p, int B, hipStream_t stream) {
  const int64_t rows = (int64_t)B * p.N;
  if (few_rows(B, p.N, p.V, p.pitch)) {
    launch_few_of<NS_FP32>(p, B, stream);
  } else if (rows <= 65536) {
    if (p.M <= 16) launch_head_stream<1, 8, 7>(p, B, stream);
    else if (p.M <= 32) launch_head_stream<2, 8, 7>(p, B, stream);
    else if (p.M <= 48) launch_head_stream<3, 8, 7>(p, B, stream);
    else launch_head_stream<4, 8, 7>(p, B, stream);
  } else {
    if (p.M <= 16) launch_head_stream<1, 16, 6>(p, B, stream);
    else if (p.M <= 32) launch_head_stream<2, 16, 6>(p, B, stream);
    else if (p.M <= 48) launch_head_stream<3, 32, 3>(p, B, stream);
    else launch_head_stream<4, 32, 3>(p, B, stream);
  }
}

// ---------------------------------------------------------------------------
// Top-k over the scaled logits of each hidden row
// ---------------------------------------------------------------------------
// Columns of a thread: 4 cover 4096 columns in one block; 16, for more, cover
// 16384 (64 x 15500: 11.5 us in chunks of 4096 with a join, 7.8 us in one).
constexpr int top_cols(int n_max) { return n_max <= 4 * kSelectThreads ? 4 : 16; }
constexpr int top_chunk(int n_max) { return kSelectThreads * top_cols(n_max); }

struct Top {
  const float* z;           // [B][M] rows, ld floats apart
  int64_t ld;
  const int32_t* ids;
  const int32_t* n_dev;
  int n_max, V, M, k;
  float* logits;            // [B][M][n_max] or NULL
  int32_t* out_ids;
  float* out_vals;
  uint64_t* cand;           // [B][M][chunks][k]
};

__device__ __forceinline__ void put_top(const Top& t, size_t row, int r, uint64_t key) {
  t.out_ids[row * t.k + r] = key ? ns::key_id(key) : -1;
  t.out_vals[row * t.k + r] = key ? ns::key_val(key) : -INFINITY;
}

// Block (m, c, b): the k best of chunk c of hidden row m of sequence b.
template <int U>
__global__ __launch_bounds__(kSelectThreads) void k_top_chunk(Top t) {
  constexpr int CHUNK = U * kSelectThreads;
  __shared__ SelectSmem sm;
  const int m = blockIdx.x, c = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const size_t row = (size_t)b * t.M + m;
  const int j0 = c * CHUNK;
  int n = t.n_dev ? t.n_dev[b] : t.n_max;
  // Every column is asked for before the first is looked at; the first four of
  // a thread together with the count, live or not.
  float val[U];
  int id[U];
  const auto ask = [&](int u, int end) {
    const int q = j0 + tid + u * kSelectThreads, j = q < end ? q : end - 1;
    val[u] = t.z[row * (size_t)t.ld + j];
    id[u] = t.ids ? t.ids[(size_t)b * t.n_max + j] : j;
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) ask(u, t.n_max);
  NS_ISSUE_FENCE();
  n = n < 0 ? 0 : (n > t.n_max ? t.n_max : n);
  const bool final_here = n <= CHUNK;
  if (final_here && c > 0) return;
  const int lim = n - j0 < CHUNK ? n - j0 : CHUNK;       // <= 0 where nothing is live
  if (U > 4) {
    const int end = n > 0 ? n : 1;
#pragma unroll
    for (int u = 4; u < U; ++u) ask(u, end);
    NS_ISSUE_FENCE();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int q = tid + u * kSelectThreads;
    const bool live = q < lim && id[u] >= 0 && id[u] < t.V;
    if (live && t.logits) t.logits[row * (size_t)t.n_max + j0 + q] = val[u];
    if (!live || val[u] != val[u]) {                     // NaN is never selected
      val[u] = 0.f;
      id[u] = -1;
    }
  }
  const int nlive = lim > 0 ? lim : 0;
  if (final_here)
    block_select_topk<U>(val, id, t.k, nlive, sm, [&](int r, uint64_t x) { put_top(t, row, r, x); });
  else {
    uint64_t* dst = t.cand + (row * gridDim.y + c) * (size_t)t.k;
    block_select_topk<U>(val, id, t.k, nlive, sm, [&](int r, uint64_t x) { dst[r] = x; });
  }
}

// Block (m, b): the k best of the nk = chunks * k keys of its chunks.
template <int U>
__global__ __launch_bounds__(kSelectThreads) void k_top_keys(Top t, int nk) {
  __shared__ SelectSmem sm;
  const int m = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  int n = t.n_dev ? t.n_dev[b] : t.n_max;
  if (n > t.n_max) n = t.n_max;
  if (n <= top_chunk(t.n_max)) return;
  const size_t row = (size_t)b * t.M + m;
  float val[U];
  int id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int q = tid + u * kSelectThreads;
    const uint64_t key = q < nk ? t.cand[row * nk + q] : 0;
    val[u] = key ? ns::key_val(key) : 0.f;
    id[u] = key ? ns::key_id(key) : -1;
  }
  block_select_topk<U>(val, id, t.k, nk, sm, [&](int r, uint64_t x) { put_top(t, row, r, x); });
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
  w.z = w.scale + align256(rows * 4);
  w.cand = w.z + align256(rows * (size_t)w.ld * 4);
  w.bytes = w.cand + (w.chunks > 1 ? align256(rows * w.chunks * (size_t)k * 8) : 0);
  return w;
}

constexpr int64_t kMaxLd = (int64_t)1 << 40;       // no product with a row count overflows

bool known_dtype(int t) { return t == NS_BF16 || t == NS_FP32 || t == NS_FP16; }
bool aligned16(const void* p) { return (((uintptr_t)p) & 15u) == 0; }

bool head_dims_ok(int B, int n_max, int M, int k, int d) {
  return B >= 1 && B <= NS_MAX_BATCH && n_max >= 1 && n_max <= NS_MAX_V && M >= 1 && M <= NS_MAX_M && k >= 1 &&
         k <= NS_MAX_K && d >= 1 && d <= NS_MAX_D;
}

}  // namespace

extern "C" {

int32_t nanospec_quant_pitch(int32_t d) { return d < 1 || d > NS_MAX_D ? 0 : pitch_of(d); }

int nanospec_quant_rows(const void* x, int64_t ld, int32_t R, int32_t d, int32_t dtype, int8_t* q, float* scale,
                        hipStream_t stream) {
  if (!known_dtype(dtype)) return NS_EDTYPE;
  if (R < 0 || R > NS_MAX_ROWS || d < 1 || d > NS_MAX_D || ld < d || ld > kMaxLd) return NS_EINVAL;
  if (R == 0) return NS_OK;
  if (!x || !q || !scale || !aligned16(q)) return NS_EINVAL;
  if (((uintptr_t)x) % (dtype == NS_FP32 ? 4 : 2)) return NS_EINVAL;
  (void)hipGetLastError();
  return quant_rows(x, ld, R, d, dtype, q, scale, stream);
}

int nanospec_quant_matmul(const int8_t* xq, const float* xs, int32_t M, const int8_t* wq, const float* ws, int32_t N,
                          int32_t d, void* out, int64_t ld_out, int32_t out_dtype, hipStream_t stream) {
  if (!known_dtype(out_dtype)) return NS_EDTYPE;
  if (M < 0 || M > NS_MAX_ROWS || N < 1 || N > NS_MAX_V || d < 1 || d > NS_MAX_D || ld_out < N ||
      ld_out > kMaxLd)
    return NS_EINVAL;
  if (M == 0) return NS_OK;
  if (!xq || !xs || !wq || !ws || !out || !aligned16(xq) || !aligned16(wq)) return NS_EINVAL;
  if (((uintptr_t)out) % (out_dtype == NS_FP32 ? 4 : 2)) return NS_EINVAL;
  (void)hipGetLastError();
  const Product p{xq, xs, wq, ws, nullptr, nullptr, M, N, N, pitch_of(d), out, ld_out, 1};
  if (out_dtype == NS_FP32) launch_product<NS_FP32>(p, stream);
  else if (out_dtype == NS_BF16) launch_product<NS_BF16>(p, stream);
  else launch_product<NS_FP16>(p, stream);
  return ns_launch_status();
}

size_t nanospec_quant_logits_workspace_bytes(int32_t B, int32_t n_max, int32_t M, int32_t k, int32_t d) {
  return head_dims_ok(B, n_max, M, k, d) ? head_ws(B, n_max, M, k, d).bytes : 0;
}

int nanospec_quant_logits_topk(const int8_t* wq, const float* wscale, const int32_t* row_ids, const int32_t* n_dev,
                               int32_t n_max, int32_t B, int32_t V, int32_t d, const void* h, int32_t dtype, int32_t M,
                               int32_t k, float* logits, int32_t* topk_ids, float* topk_vals, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
  if (!known_dtype(dtype)) return NS_EDTYPE;
  if (!head_dims_ok(B, n_max, M, k, d) || V < 1 || V > NS_MAX_V || (!row_ids && n_max > V)) return NS_EINVAL;
  if (!wq || !wscale || !h || !topk_ids || !topk_vals || !ws) return NS_EINVAL;
  if (!aligned16(wq) || (((uintptr_t)ws) & 255u) || ((uintptr_t)h) % (dtype == NS_FP32 ? 4 : 2)) return NS_EINVAL;
  const HeadWs l = head_ws(B, n_max, M, k, d);
  if (ws_bytes < l.bytes) return NS_ECAPACITY;
  (void)hipGetLastError();
  char* base = (char*)ws;
  int8_t* hq = (int8_t*)(base + l.q);
  float* hs = (float*)(base + l.scale);
  float* z = (float*)(base + l.z);
  int rc = NS_OK;
  const bool fused = few_rows(B, n_max, V, d) && M <= 16 && M * pitch_of(d) <= kFusedBytes && d % 8 == 0;
  if (!fused) rc = quant_rows(h, d, B * M, d, dtype, hq, hs, stream);
  if (rc != NS_OK) return rc;
  const Product p{hq, hs, wq, wscale, row_ids, n_dev, M, n_max, V, pitch_of(d), z, l.ld, 1};
  if (!fused) {
    launch_head(p, B, stream);
  } else {
    if (dtype == NS_BF16) launch_head_few<NS_BF16>(p, B, h, d, stream);
    else if (dtype == NS_FP16) launch_head_few<NS_FP16>(p, B, h, d, stream);
    else launch_head_few<NS_FP32>(p, B, h, d, stream);
  }
  rc = ns_launch_status();
  if (rc != NS_OK) return rc;
  const Top t{z, l.ld, row_ids, n_dev, n_max, V, M, k, logits, topk_ids, topk_vals, (uint64_t*)(base + l.cand)};
  const dim3 chunks((unsigned)M, (unsigned)l.chunks, (unsigned)B);
  if (top_cols(n_max) == 4) hipLaunchKernelGGL(k_top_chunk<4>, chunks, dim3(kSelectThreads), 0, stream, t);
  else hipLaunchKernelGGL(k_top_chunk<16>, chunks, dim3(kSelectThreads), 0, stream, t);
  rc = ns_launch_status();
  if (rc != NS_OK || l.chunks == 1) return rc;
  const int nk = l.chunks * k;
  const dim3 grid((unsigned)M, (unsigned)B), block(kSelectThreads);
  static_assert((NS_MAX_V + top_chunk(NS_MAX_V) - 1) / top_chunk(NS_MAX_V) * NS_MAX_K <= 4 * kSelectThreads,
                "k_top_keys<4> holds every chunk's keys");
  if (nk <= kSelectThreads) hipLaunchKernelGGL(k_top_keys<1>, grid, block, 0, stream, t, nk);
  else hipLaunchKernelGGL(k_top_keys<4>, grid, block, 0, stream, t, nk);
  return ns_launch_status();
}

}  // extern "C"
