// The experts' products and their gradients: matrix products on the matrix
// cores, one launch for the experts of all ranks.
//
//   forward       out[s][f]    = act(Σ_h x[s][h]·W_e[f][h] + b_e[f]) + residual[s][f]
//   rows' grad    dx[s][h]     = Σ_f dz[s][f]·W_e[f][h]
//   weights' grad dW_e[f][h]   = Σ_s dz[s][f]·x[s][h]      over the rows s of expert e
//
// Each is C[m][n] = Σ_k A[m,k]·B[n,k] with one of two layouts per operand:
// "along" (k runs along memory: x, dz and W in the forward product) and
// "across" (k strides: W for the rows' gradient, both operands of the
// weights' gradient).
//
// A workgroup computes a tile of C in stages of 128 bytes of k (64 bf16 or 32
// float32: whole lines of an operand along k), of two halves each.  LDS
// holds two stages.  While the waves multiply one half out of registers,
// they read the fragments of the next half from LDS, and the loads of the
// stage after next are on their way from memory straight into LDS (buffer
// loads to LDS, 16 bytes a lane, no registers in between).  One barrier per
// stage orders it all, between its halves: before it a wave waits for its
// fragment reads of the second half and for its loads of the next stage, so
// behind it the next stage is whole, and this stage's buffer, now in
// everyone's registers, may be overwritten.  The buffer resource of a load
// ends where the operand's valid range ends, so what lies behind it reads as
// zero; a lane whose k lies behind the end of k asks for an address beyond
// the resource.
//
// LDS writes of such a load are consecutive in lane order, so padding is not
// possible; instead each lane picks which 16-byte chunk of the row it
// fetches, chunk XOR key(row), with the key chosen such that the fragment
// reads of a wave spread over the banks.
//
// Fragments.  The 16x16 matrix instructions take, from lane l, row l % 16
// and the k group l / 16 of each operand.  "Along" fragments are one 16-byte
// LDS read.  "Across" fragments of bf16 use the transposing LDS read (16
// lanes read 4 rows of 16 elements and each gets one column of 4), those of
// float32 read element by element.  In float32 a lane's 16 bytes are 4
// consecutive k, so instruction s of four takes k = 4·group + s in both
// operands: a permutation of k, which a sum does not see.
//
// The instruction is issued with the operands swapped, so a lane ends up
// with 4 consecutive n of one row m per fragment; and the n fragments of a
// wave interleave such that fragment j covers n = 16·i + 4·j + (0..3), i =
// 0..3, of the wave's 64 columns.  A lane then holds 16 consecutive n of a
// row: the bias, the residual and the stores move whole 16-byte vectors,
// four lanes a 128-byte line.

#include <cstdio>

#include "experts.hpp"
#include "kernel_common.hpp"

namespace ccl {
namespace {

#define CCL_LDS __attribute__((address_space(3)))

constexpr int kWave = 64;
constexpr int kStageBytes = 128;  // k bytes of one stage
constexpr int kWaveN = 64;        // columns of a wave's part of the tile

__device__ inline int lane_id() { return static_cast<int>(threadIdx.x) & (kWave - 1); }
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave); }

// The same value, which the compiler works out again at each use instead of
// keeping what follows from it in registers through the loops.
__device__ inline uint32_t afresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

enum Mode : int { kForward = 0, kGradRows = 1, kGradWeights = 2 };

struct ProductArgs {
  RankPtrs a, b, offsets, out, bias, residual, preact;
  // An operand in the workspace, the ranks' parts `step` bytes apart; else NULL.
  const char *a_at, *b_at;
  uint64_t a_step, b_step;
  float* parts;          // weights' gradient of several splits: float32 sums, [splits][nranks][per_rank][m][n]
  uint32_t nranks, per_rank, capacity;
  uint32_t m, n, k;      // features and hidden as the mode uses them; m / k of the ragged axis unused
  uint32_t lda, ldb;     // row strides of the operands, in elements
  uint32_t splits;       // parts of k (weights' gradient)
  uint32_t least;        // forward: experts with fewer rows are the form's for few rows (0: none are)
  uint32_t ntiles;       // tiles of n
  bool has_offsets, has_bias, has_residual, has_preact;
  int activation;
};

// ---------------------------------------------------------------------------
// Which rows an expert has, and which expert a tile belongs to.
// ---------------------------------------------------------------------------
struct Range {
  uint32_t expert, lo, hi;  // expert = per_rank: none
  uint32_t tile;            // tile within the expert
};

// One offset, cut to [0, capacity].
__device__ inline uint32_t offset_at(const int* off, uint32_t e, uint32_t capacity) {
  const int v = get1(off + e);
  return v < 0 ? 0u : (uint32_t(v) < capacity ? uint32_t(v) : capacity);
}

// The rows of expert e; none when there are fewer than `least`.
__device__ inline Range rows_of(const int* off, uint32_t e, uint32_t capacity, uint32_t least = 0) {
  Range r{e, 0, capacity, 0};
  if (off != nullptr) {
    r.lo = offset_at(off, e, capacity);
    r.hi = offset_at(off, e + 1, capacity);
  }
  if (r.hi < r.lo || r.hi - r.lo < least) r.hi = r.lo;
  return r;
}

// The expert whose rows hold tile `slot` when every expert's rows are cut
// into tiles of `rows` of their own, found by the whole wave: 64 experts at
// a time, a scan over the lanes' tile counts.
__device__ inline Range find_tile(const int* off, uint32_t per_rank, uint32_t capacity, uint32_t slot, uint32_t rows,
                                  uint32_t least = 0) {
  if (off == nullptr) return Range{slot * uint64_t(rows) < capacity ? 0u : per_rank, 0, capacity, slot};
  uint32_t before = 0;
  const uint32_t lane = afresh(uint32_t(lane_id()));
  for (uint32_t e0 = 0; e0 < per_rank; e0 += kWave) {
    const uint32_t e = e0 + lane;
    Range r{e, 0, 0, 0};
    if (e < per_rank) r = rows_of(off, e, capacity, least);
    const uint32_t n = (r.hi - r.lo + rows - 1) / rows;
    uint32_t incl = n;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const uint32_t u = uint32_t(__shfl_up(int(incl), d));
      if (lane >= uint32_t(d)) incl += u;
    }
    const uint64_t past = __ballot(before + incl > slot);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      Range f;
      f.expert = e0 + uint32_t(l);
      f.lo = uint32_t(__builtin_amdgcn_readlane(int(r.lo), l));
      f.hi = uint32_t(__builtin_amdgcn_readlane(int(r.hi), l));
      f.tile = slot - (before + uint32_t(__builtin_amdgcn_readlane(int(incl - n), l)));
      return f;
    }
    before += uint32_t(__builtin_amdgcn_readlane(int(incl), kWave - 1));
  }
  return Range{per_rank, 0, 0, 0};
}

// ---------------------------------------------------------------------------
// Activations, in float32.
//
// float32 calls the library's functions and divides.  bf16, whose result
// keeps 8 bits, takes the hardware's exponential and reciprocal (each off by
// a step of float32 or so) and a polynomial for the normal distribution's
// tail: 128 values a lane go through this at the end of a tile, while the
// matrix units wait, and the library's functions took four times as long (the
// gradient's pass over 2,900 rows of 1736, GELU: 27 us, now 14).
//
// Both take Φ from its tail, not from 1 + erf, which loses all of its bits
// far on the negative side (float32: 5 % at z = -4.5, everything from -5.6
// on).  The tail of bf16 is Φ(-√2·x) = e^(-x²)·t·P(t) with t = 1 / (1 +
// 0.375·x); P was fitted to e^(x²)·erfc(x) / 2 over x = 0 to 10 for the
// smallest largest relative error (a linear program over 1,500 points), which
// is 6e-7.
// ---------------------------------------------------------------------------
template <class T>
constexpr bool kExactActivation = sizeof(typename T::S) == 4;

__device__ inline float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ inline float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + e^-z)
template <class T>
__device__ inline float sigmoid(float z) {
  if constexpr (kExactActivation<T>) return 1.0f / (1.0f + expf(-z));
  else return fast_rcp(1.0f + fast_exp(-z));
}

// Φ(z), and e^(-z²/2) for the derivative.
template <class T>
__device__ inline float normal_cdf(float z, float* gauss) {
  if constexpr (kExactActivation<T>) {
    *gauss = expf(-0.5f * z * z);
    return 0.5f * erfcf(z * -0.70710678f);
  } else {
    const float x = fabsf(z) * 0.70710678f, t = fast_rcp(1.0f + 0.375f * x);
    const float poly =
        t * (0.105670191f + t * (0.107838698f + t * (0.0833611116f + t * (0.141461387f + t * (-0.0647118539f + t * (0.193915024f + t * -0.0675348565f))))));
    *gauss = fast_exp(-x * x);
    const float tail = poly * *gauss;  // Φ(-|z|)
    return z < 0.0f ? tail : 1.0f - tail;
  }
}

template <class T>
__device__ inline float activate(float z, int act) {
  float gauss;
  switch (act) {
    case CCL_SIM_ACT_RELU: return z < 0.0f ? 0.0f : z;  // a NaN stays one
    case CCL_SIM_ACT_GELU: return z * normal_cdf<T>(z, &gauss);
    case CCL_SIM_ACT_SILU:
      if constexpr (kExactActivation<T>) return z / (1.0f + expf(-z));
      else return z * sigmoid<T>(z);
    default: return z;
  }
}

// The derivative at z.  SiLU's is σ(1 + z(1 - σ)).
template <class T>
__device__ inline float slope(float z, int act) {
  float gauss;
  switch (act) {
    case CCL_SIM_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case CCL_SIM_ACT_GELU: {
      const float cdf = normal_cdf<T>(z, &gauss);
      return cdf + z * 0.39894228f * gauss;
    }
    case CCL_SIM_ACT_SILU: {
      const float s = sigmoid<T>(z);
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

// ---------------------------------------------------------------------------
// Operand tiles in LDS.
//   along:  [rows of m or n][128 bytes of k]
//   across: [k][WIDTH elements of m or n]
// ---------------------------------------------------------------------------
template <class S>
struct Elem {
  static constexpr int kSize = int(sizeof(S));
  static constexpr int kStage = kStageBytes / kSize;  // k elements of a stage
  static constexpr int kChunk = 16 / kSize;           // elements of a 16-byte chunk
};

// Chunk permutation of a row.  PERM: the operand's rows are read in the
// interleaved order of the n fragments (lanes i = 0..15 read rows
// 16·(i/4) + 4·j + i%4), else consecutively.  Along: 8 consecutive lanes of a
// fragment read then fall on the 8 different chunk positions of a row.
template <class S, bool ACROSS, bool PERM, int WIDTH>
__device__ inline uint32_t key_of(uint32_t row) {
  if constexpr (!ACROSS) {
    return PERM ? (row & 3) | ((row >> 4) & 1) << 2 : row & 7;
  } else if constexpr (sizeof(S) == 2) {
    // transposing reads: 16 k rows at once, 32 bytes (consecutive) or four
    // times 8 bytes 32 apart (interleaved) of each; a row of 64 has 8 chunks
    if constexpr (WIDTH < 128) return PERM ? (row & 1) | (row & 2) << 1 : (row & 3) << 1;
    return PERM ? (row & 1) | (row & 2) << 2 : ((row & 3) | ((row >> 3) & 1) << 2) << 1;
  } else {
    return PERM ? (row >> 2) & 3 : ((row >> 2) & 3) << 2;
  }
}

// A value that is the same in every lane, in a scalar register.
__device__ inline uint32_t uniform(uint32_t v) { return uint32_t(__builtin_amdgcn_readfirstlane(int(v))); }

// One 16-byte load per lane from a buffer straight into LDS: lane l's lands
// at lds + 16·l.  In assembly, since the compiler orders every later LDS read
// behind such a load it knows of; here the waits are the kernel's own.  The
// instruction has no register result; m0 holds the LDS address.  m0 is
// reserved: the compiler keeps no value of its own in it (and refuses it as a
// clobber), and a test of the assembly holds that nothing else here uses it.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t rs, uint32_t lds, uint32_t offset, uint32_t more) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(uniform(lds)), "v"(offset), "s"(rs), "s"(uniform(more))
      : "memory");
}
__device__ inline uint32_t lds_address(const char* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((const CCL_LDS char*)p));
}

template <class S, bool ACROSS, bool PERM, int WIDTH, int THREADS>
struct Tile {
  using El = Elem<S>;
  static constexpr int kBytes = WIDTH * kStageBytes;
  static constexpr int kLoads = kBytes / (THREADS * 16);         // loads of a lane per stage
  static constexpr int kRowBytes = ACROSS ? WIDTH * El::kSize : kStageBytes;
  static constexpr int kRowChunks = kRowBytes / 16;
  static_assert(kBytes % (THREADS * 16) == 0);

  // Position of this lane's load q of a stage, and the chunk it fetches.
  __device__ static uint32_t linear(int q, uint32_t t = threadIdx.x) { return uint32_t(q) * THREADS + t; }
  __device__ static uint32_t row_of(int q, uint32_t t = threadIdx.x) { return linear(q, t) / kRowChunks; }
  __device__ static uint32_t chunk_of(int q, uint32_t t = threadIdx.x) {
    return (linear(q, t) % kRowChunks) ^ key_of<S, ACROSS, PERM, WIDTH>(row_of(q, t));
  }

  // Loads straight to LDS: what a wave needs for them, worked out once.  A
  // stage then costs a few scalar operations.
  //   along:  the resource starts at the tile's first row and ends with the
  //           last valid one; a stage adds its k offset (scalar, and part of
  //           the range check).
  //   across: the resource starts at the stage's first row of k, which moves
  //           on by a 64-bit address, and ends with the stage's last valid one.
  // In the last stage, and behind the end of k, lanes whose k is past the end
  // (along) or rows past it (across) ask behind the resource.
  //
  // A lane's loads of a stage lie kRowStep rows apart, which leaves the chunk
  // permutation as it is (float32 across: in every second one), so one place
  // per lane (two) serves all of them.
  static constexpr int kRowStep = THREADS / kRowChunks;
  static constexpr int kPlaces = ACROSS && El::kSize == 4 ? 2 : 1;
  static_assert(kRowStep % (kPlaces == 2 ? 8 : !ACROSS ? 32 : 16) == 0 || kLoads == 1);
  struct Direct {
    const char* base = nullptr;
    uint32_t bytes = 0;       // along: of the valid rows; across: of a whole stage's rows
    uint32_t row, lds;        // bytes of a row; this wave's part of a stage in LDS
    uint32_t place[kPlaces];  // this lane's places

    // `ld`: row stride in elements.
    __device__ explicit Direct(uint32_t ld) {
      row = ld * El::kSize;
      lds = uint32_t(wave_id()) * kWave * 16;
#pragma unroll
      for (int q = 0; q < kPlaces; ++q) place[q] = (row_of(q) - q * kRowStep) * row + chunk_of(q) * 16;
    }
    // `at`: the tile's first element at k = 0; `rows`: valid rows from there
    // (along), or the elements of a row before the tile (across).
    __device__ void set(const S* at, uint32_t rows) {
      base = reinterpret_cast<const char*>(at);
      const uint64_t all = ACROSS ? uint64_t(El::kStage) * row - rows * El::kSize : uint64_t(rows) * row;
      bytes = uniform(all < 0x7FFFFFF0ull ? uint32_t(all) : 0x7FFFFFF0u);
    }
    // `buffer`: LDS address of the stage's tile.
    __device__ void load(uint32_t buffer, uint32_t k0, uint32_t k) const {
      const bool whole = k0 + El::kStage <= k;
      uint32_t records = bytes, more = ACROSS ? 0 : k0 * El::kSize;
      if constexpr (ACROSS)
        if (!whole) records = k0 < k ? bytes - (El::kStage - (k - k0)) * row : 0;
      const __amdgpu_buffer_rsrc_t rs = tile_rsrc(ACROSS ? base + uint64_t(k0) * row : base, uniform(records));
      uint32_t at[kPlaces];
#pragma unroll
      for (int q = 0; q < kPlaces; ++q) {
        at[q] = place[q];
        if constexpr (!ACROSS)
          if (!whole && k0 + chunk_of(q, afresh(threadIdx.x)) * El::kChunk >= k) at[q] = 0x7FFFFFFFu;
      }
#pragma unroll
      for (int q = 0; q < kLoads; ++q)
        load_to_lds(rs, buffer + lds + uint32_t(q) * THREADS * 16, at[q % kPlaces], more + uint32_t(q) * kRowStep * row);
    }
  };

  // The same through registers, for layouts whose rows do not start on 16
  // bytes or whose ends cut a chunk: whole chunks as one unaligned load,
  // cut ones element by element.  `cols`: valid columns from the base (across).
  using Chunk = typename VecOf<S, El::kChunk>::type;
  __device__ static void load_regs(Chunk* v, const S* base, uint32_t ld, uint32_t rows, uint32_t k0, uint32_t k,
                                   uint32_t cols) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const uint32_t r = row_of(q), c = chunk_of(q) * El::kChunk;
      const uint32_t row_end = ACROSS ? (k0 < k ? k - k0 : 0) : rows, col = ACROSS ? c : k0 + c, col_end = ACROSS ? cols : k;
      const uint64_t row = ACROSS ? uint64_t(k0) + r : r;
      v[q] = Chunk{};
      if (r >= row_end || col >= col_end) continue;
      const S* p = base + row * ld + col;
      if (col + El::kChunk <= col_end) {
        v[q] = vload<S, El::kChunk, false>(p);
      } else {
#pragma unroll
        for (int i = 0; i < El::kChunk; ++i)
          if (col + i < col_end) v[q][i] = get1(p + i);
      }
    }
  }
  __device__ static void store_regs(char* lds, const Chunk* v) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      *(CCL_LDS W4*)(CCL_LDS char*)(lds + linear(q) * 16) = __builtin_bit_cast(W4, v[q]);
  }
};

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef short short8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));

// Fragment reads of one operand.  A lane's address of fragment f in half
// `half` (64 bytes of k) of a stage is a sum of `row`, a constant, and
// `chunk` XOR a constant; the two lane values are worked out once.  `first`:
// the wave's first row or column in the tile, a multiple of what the wave
// takes, so that it, the lane's and the fragment's parts of a chunk number
// have no bit in common.
template <class S, bool ACROSS, bool PERM, int WIDTH>
struct Reader {
  static constexpr uint32_t kRowBytes = ACROSS ? WIDTH * sizeof(S) : kStageBytes;
  uint32_t row, chunk;

  __device__ explicit Reader(uint32_t first) {
    const uint32_t l = uint32_t(lane_id()), i = l % 16, g = l / 16;
    if constexpr (!ACROSS) {
      const uint32_t r = first + (PERM ? 16 * (i / 4) + i % 4 : i);
      row = r * kRowBytes;
      chunk = (g ^ key_of<S, false, PERM, WIDTH>(r)) * 16;
    } else if constexpr (sizeof(S) == 2) {
      const uint32_t k = g * 8 + i / 4;
      row = k * kRowBytes + (PERM ? 0 : i % 2 * 8);
      chunk = ((first / 8) ^ (PERM ? i % 4 * 2 : i % 4 / 2) ^ key_of<S, true, PERM, WIDTH>(k)) * 16;
    } else {
      const uint32_t k = g * 4;
      row = k * kRowBytes + i % 4 * 4;
      chunk = ((first / 4) ^ (PERM ? i / 4 * 4 : i / 4) ^ key_of<S, true, PERM, WIDTH>(k)) * 16;
    }
  }

  // From a copy with the buffer's offset added (see `at`).
  __device__ float4_t read(const char* lds, int f, int half) const {
    if constexpr (!ACROSS) {
      const uint32_t a = row + (chunk ^ uint32_t(half * 64)) + uint32_t(f) * (PERM ? 4 : 16) * kRowBytes;
      return *(const CCL_LDS float4_t*)(const CCL_LDS char*)(lds + a);
    } else if constexpr (sizeof(S) == 2) {
      const uint32_t a = row + (chunk ^ uint32_t(PERM ? f / 2 * 16 : f * 32)) + (PERM ? f % 2 * 8 : 0) +
                         uint32_t(half) * 32 * kRowBytes;
      short4_t h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (CCL_LDS short4_t*)(CCL_LDS char*)const_cast<char*>(lds + a + uint32_t(u) * 4 * kRowBytes));
      const short8_t v = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(float4_t, v);
    } else {
      const uint32_t a = row + (chunk ^ uint32_t(f * (PERM ? 16 : 64))) + uint32_t(half) * 16 * kRowBytes;
      float4_t v;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        v[s] = *(const CCL_LDS float*)(const CCL_LDS char*)(lds + a + uint32_t(s) * kRowBytes);
      return v;
    }
  }
  // This reader in the buffer at `offset`; a register of its own for every
  // fragment's address would be more than there are.
  __device__ Reader at(uint32_t offset) const {
    Reader r = *this;
    r.row = afresh(row + offset);
    r.chunk = afresh(chunk);
    return r;
  }
};

// acc += B fragment · A fragment (swapped: rows of the result are n).
template <class T>
__device__ inline float4_t multiply(float4_t b, float4_t a, float4_t acc) {
  if constexpr (sizeof(typename T::S) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b), __builtin_bit_cast(bf16x8_t, a), acc,
                                                   0, 0, 0);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(b[s], a[s], acc, 0, 0, 0);
    return acc;
  }
}

// Up to 16 bytes from element k on of a row that ends at `end`: zeros behind it.
template <class S, bool NT = false>
__device__ inline typename VecOf<S, 16 / int(sizeof(S))>::type cut(const S* p, uint32_t k, uint32_t end) {
  constexpr int V = 16 / int(sizeof(S));
  if (k + V <= end) return vload<S, V, NT>(p);
  typename VecOf<S, V>::type v = {};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (k + uint32_t(i) < end) v[i] = get1(p + i);
  return v;
}

// float32 to the stored type, to nearest even; one instruction for two bf16.
template <class T>
__device__ inline typename T::S round_to(float v) {
  if constexpr (sizeof(typename T::S) == 2) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else return v;
}

// 16 consecutive elements of a row from column n0 on, as float32.
template <class T>
__device__ inline void load16(float* v, const typename T::S* p, uint32_t n0, uint32_t n) {
  using S = typename T::S;
  constexpr int V = 16 / int(sizeof(S));
  if (n0 + 16 <= n) {
#pragma unroll
    for (int u = 0; u < 16 / V; ++u) {
      const auto x = vload<S, V, false>(p + u * V);
#pragma unroll
      for (int i = 0; i < V; ++i) v[u * V + i] = T::widen(x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = n0 + uint32_t(i) < n ? T::widen(get1(p + i)) : 0.0f;
  }
}
template <class T, bool NT = false>
__device__ inline void store16(typename T::S* p, const float* v, uint32_t n0, uint32_t n) {
  using S = typename T::S;
  constexpr int V = 16 / int(sizeof(S));
  if (n0 + 16 <= n) {
#pragma unroll
    for (int u = 0; u < 16 / V; ++u) {
      typename VecOf<S, V>::type x;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = round_to<T>(v[u * V + i]);
      vstore<S, V, NT>(p + u * V, x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n0 + uint32_t(i) < n) put1(p + i, round_to<T>(v[i]));
  }
}

// ---------------------------------------------------------------------------
// The tile kernel.  MF fragments of m per wave, WM x WN waves: a tile of
// 16·MF·WM rows and 64·WN columns.
//
// Bound by the matrix units and, at full rate on all of them, by the clock
// that the power leaves: on 8192^3 the units are busy in two thirds of the
// cycles and the clock falls to 1.9 GHz.  256 x 256 tiles by 8 waves reach
// 1,300-1,430 TFLOP/s there in bf16, by layout (the library's product 1,090
// to 1,384); 4 waves of 128 x 128 each, and two workgroups of 128 x 256 per
// compute unit, reached 1,250 and 950; three or four stages in LDS instead of
// two gained nothing, since a second workgroup fits no more.  Workgroups stay
// and take tile after tile (8 ranks of 4,096 rows, 2560 -> 5120: 978 to 1,035
// TFLOP/s).
// ---------------------------------------------------------------------------
template <class T, int MODE, bool DIRECT, int MF, int WM, int WN>
__global__ __launch_bounds__(WM* WN* kWave, 2) void product_kernel(ProductArgs a) {
  using S = typename T::S;
  using El = Elem<S>;
  constexpr int kThreads = WM * WN * kWave;
  constexpr int BM = 16 * MF * WM, BN = kWaveN * WN, NF = 4;
  constexpr bool kAAcross = MODE == kGradWeights, kBAcross = MODE != kForward;
  using TA = Tile<S, kAAcross, false, BM, kThreads>;
  using TB = Tile<S, kBAcross, true, BN, kThreads>;
  constexpr int kStage = TA::kBytes + TB::kBytes;
  __shared__ __attribute__((aligned(128))) char lds[2 * kStage];
  __shared__ uint32_t rank_tiles[MODE == kGradWeights ? 1 : CCL_SIM_MAX_RANKS + 1];

  // Which tiles a workgroup computes.  Consecutive workgroups land on
  // different XCDs, each with its own L2; every XCD takes a consecutive run
  // of tiles, in an order that walks all of m for kGroup tiles of n, whose
  // weights stay in that L2 meanwhile.
  //   ragged m:  the tiles that there are, of all ranks, counted here from
  //              the offsets; a run per XCD, its workgroups taking turns.
  //   weights' gradient: every XCD takes an eighth of each expert's tiles (an
  //              expert's tiles all have its k, and experts differ in it),
  //              one workgroup a tile, or taking turns where a launch cannot
  //              hold as many.
  constexpr uint32_t kGroup = 4;
  const uint32_t xcd = blockIdx.x & 7, turn = blockIdx.x >> 3;
  const uint32_t lda = a.lda, ldb = a.ldb;
  uint32_t unit = 0, unit_end = 0;
  if constexpr (MODE != kGradWeights) {
    for (uint32_t r = threadIdx.x; r <= a.nranks; r += kThreads) rank_tiles[r] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.nranks * a.per_rank; i += kThreads) {
      const uint32_t r = i / a.per_rank;
      const int* off = a.has_offsets ? static_cast<const int*>(a.offsets.get(int(r))) : nullptr;
      const Range e = rows_of(off, i - r * a.per_rank, a.capacity, a.least);
      if (e.hi > e.lo) atomicAdd(&rank_tiles[r + 1], (e.hi - e.lo + BM - 1) / BM);
    }
    __syncthreads();
    if (wave_id() == 0) {  // inclusive sums over the ranks
      uint32_t before = 0;
      for (uint32_t r0 = 0; r0 < a.nranks; r0 += kWave) {
        const uint32_t r = r0 + uint32_t(lane_id());
        uint32_t v = r < a.nranks ? rank_tiles[r + 1] : 0;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
          const uint32_t u = uint32_t(__shfl_up(int(v), d));
          if (lane_id() >= d) v += u;
        }
        if (r < a.nranks) rank_tiles[r + 1] = before + v;
        before += uint32_t(__shfl(int(v), kWave - 1));
      }
    }
    __syncthreads();
    const uint64_t total = uint64_t(uniform(rank_tiles[a.nranks])) * a.ntiles;
    unit = uint32_t(total * xcd / 8) + turn;
    unit_end = uint32_t(total * (xcd + 1) / 8);
  } else {
    const uint32_t tiles = (a.m + BM - 1) / BM * a.ntiles;
    unit = turn;
    unit_end = a.nranks * a.per_rank * a.splits * ((tiles + 7) / 8);
  }

  // One tile.  m and k count from the expert's first row where they are its
  // rows.
  struct Job {
    uint32_t rank, expert, lo, rows;  // the expert's first row and their number
    uint32_t m0, n0, split;
    bool on;                          // there is a tile
  };
  auto m_end = [&](const Job& j) { return MODE == kGradWeights ? a.m : j.rows; };
  auto k_end = [&](const Job& j) { return MODE == kGradWeights ? j.rows : a.k; };
  auto next_job = [&]() -> Job {
    Job j{};
    if (unit >= unit_end) return j;
    uint32_t mtiles, rest, mtile;
    Range r;
    if constexpr (MODE != kGradWeights) {
      // the last rank whose tiles start at or before the unit
      uint32_t rank = 0;
      for (uint32_t r0 = 0; r0 < a.nranks; r0 += kWave) {
        const uint32_t q = r0 + afresh(uint32_t(lane_id()));
        const uint64_t past = __ballot(q < a.nranks && uint64_t(rank_tiles[q + 1]) * a.ntiles > unit);
        if (past != 0) {
          rank = r0 + uint32_t(__builtin_ctzll(past));
          break;
        }
      }
      const uint32_t first = uniform(rank_tiles[rank]);
      mtiles = uniform(rank_tiles[rank + 1]) - first;
      rest = unit - first * a.ntiles;
      j.rank = rank;
    } else {
      mtiles = (a.m + BM - 1) / BM;
      const uint32_t tiles = mtiles * a.ntiles, slots = (tiles + 7) / 8;
      uint32_t q;
      for (;; unit += gridDim.x >> 3) {  // over the slots that an eighth of few tiles leaves empty
        if (unit >= unit_end) return j;
        q = unit / slots;
        const uint32_t part = (xcd + q) & 7;
        rest = tiles * part / 8 + (unit - q * slots);
        if (rest < tiles * (part + 1) / 8) break;
      }
      j.split = q % a.splits;
      j.rank = q / a.splits / a.per_rank;
      j.expert = q / a.splits - j.rank * a.per_rank;
    }
    unit += gridDim.x >> 3;
    const uint32_t ngroup = rest / (mtiles * kGroup);
    rest -= ngroup * mtiles * kGroup;
    const uint32_t wide = a.ntiles - ngroup * kGroup < kGroup ? a.ntiles - ngroup * kGroup : kGroup;
    mtile = rest / wide;
    j.n0 = (ngroup * kGroup + rest % wide) * BN;
    const int* off = a.has_offsets ? static_cast<const int*>(a.offsets.get(int(j.rank))) : nullptr;
    if constexpr (MODE == kGradWeights) {
      r = rows_of(off, j.expert, a.capacity);
    } else {
      r = find_tile(off, a.per_rank, a.capacity, mtile, BM, a.least);
      j.expert = uniform(r.expert);
      if (j.expert >= a.per_rank) return j;
      mtile = uniform(r.tile);
    }
    j.lo = uniform(r.lo);
    j.rows = uniform(r.hi) - j.lo;
    if constexpr (MODE == kGradWeights)
      if (a.splits > 1) {
        const uint32_t share = ((j.rows + a.splits - 1) / a.splits + El::kStage - 1) / El::kStage * El::kStage;
        const uint32_t skip = share * j.split < j.rows ? share * j.split : j.rows;
        j.lo += skip;
        j.rows = j.rows - skip < share ? j.rows - skip : share;
      }
    j.m0 = mtile * BM;
    j.on = true;
    return j;
  };

  const int w = wave_id(), wm = w / WN, wn = w % WN;
  float4_t acc[MF][NF];

  // Loads of a stage, into the buffers in turn.  Through registers, fetch
  // starts them and settle writes them to LDS.
  const uint32_t lds_base = uniform(lds_address(lds));
  typename TA::Direct da(lda);
  typename TB::Direct db(ldb);
  typename TA::Chunk va[DIRECT ? 1 : TA::kLoads];
  typename TB::Chunk vb[DIRECT ? 1 : TB::kLoads];
  const S *pa = nullptr, *pb = nullptr;
  uint32_t fetched = 0;  // stages so far
  auto fetch = [&](const Job& job, uint32_t stage) {
    uint32_t k0 = stage * El::kStage;
    if constexpr (MODE == kForward) {
      // Tiles start at different stages of k, and go round: with a row length
      // of few different channels (5,120 bytes, say) tiles that walk k in
      // step ask the same channels of the L2 all the time.  At most three
      // stages apart, which the L2 holds for the tiles that share an operand.
      // Measured on 8 ranks of 4,096 rows in bf16: 2560 -> 5120 1,043 to
      // 1,081 TFLOP/s, 4096 -> 4096 1,193 and 1,189; the gradients gain
      // nothing.
      const uint32_t k = k_end(job), stages = (k + El::kStage - 1) / El::kStage;
      if (stages >= 16) {
        k0 += ((job.m0 / BM + job.n0 / BN) & 3) * El::kStage;
        if (k0 >= stages * El::kStage) k0 -= stages * El::kStage;
      }
    }
    if constexpr (DIRECT) {
      const uint32_t at = lds_base + (fetched & 1) * kStage;
      da.load(at, k0, job.on ? k_end(job) : 0);
      db.load(at + TA::kBytes, k0, job.on ? k_end(job) : 0);
    } else {
      const uint32_t k = job.on ? k_end(job) : 0;
      TA::load_regs(va, pa, lda, m_end(job) - job.m0, k0, k, m_end(job) - job.m0);
      TB::load_regs(vb, pb, ldb, a.n - job.n0, k0, k, a.n - job.n0);
    }
    ++fetched;
  };
  auto settle = [&]() {
    if constexpr (!DIRECT) {
      char* la = lds + ((fetched - 1) & 1) * kStage;
      TA::store_regs(la, va);
      TB::store_regs(la + TA::kBytes, vb);
    }
  };
  // The operands' first elements of a tile.
  auto enter = [&](const Job& j) {
    const S* x = static_cast<const S*>(a.a_at ? a.a_at + j.rank * a.a_step : a.a.get(int(j.rank)));
    const S* y = static_cast<const S*>(a.b_at ? a.b_at + j.rank * a.b_step : a.b.get(int(j.rank)));
    x += MODE == kGradWeights ? uint64_t(j.lo) * lda + j.m0 : uint64_t(j.lo + j.m0) * lda;
    if constexpr (MODE == kForward) y += (uint64_t(j.expert) * a.n + j.n0) * ldb;
    if constexpr (MODE == kGradRows) y += uint64_t(j.expert) * a.k * ldb + j.n0;
    if constexpr (MODE == kGradWeights) y += uint64_t(j.lo) * ldb + j.n0;
    if constexpr (DIRECT) {
      da.set(x, kAAcross ? j.m0 : m_end(j) - j.m0);
      db.set(y, kBAcross ? j.n0 : a.n - j.n0);
    } else {
      pa = x;
      pb = y;
    }
  };
  // Waits for this wave's LDS accesses and all but the newest LEFT of its
  // loads, then for the other waves.
  auto wait_all = [&]<int LEFT>() {
    if constexpr (DIRECT)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT) : "memory");
    else
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  struct Frags {
    float4_t a[MF], b[NF];
  };
  const Reader<S, kAAcross, false, BM> read_a(uint32_t(wm) * MF * 16);
  const Reader<S, kBAcross, true, BN> read_b(uint32_t(wn) * kWaveN);
  auto read = [&](Frags& f, uint32_t stage, int half) {
    const auto ra = read_a.at((stage & 1) * kStage);
    const auto rb = read_b.at((stage & 1) * kStage + TA::kBytes);
#pragma unroll
    for (int j = 0; j < NF; ++j) f.b[j] = rb.read(lds, j, half);
#pragma unroll
    for (int i = 0; i < MF; ++i) f.a[i] = ra.read(lds, i, half);
  };
  auto products = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = multiply<T>(f.b[j], f.a[i], acc[i][j]);
    if constexpr (DIRECT && sizeof(S) == 2)
#pragma unroll
      for (int i = 0; i < MF + NF; ++i) {  // the next half's LDS reads between the products
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      }
  };

  // Epilogue: 16 consecutive columns of MF rows per lane.
  auto store = [&](const Job& job) {
    const uint32_t l = afresh(uint32_t(lane_id()));
    const uint32_t n = job.n0 + uint32_t(wn) * kWaveN + (l / 16) * 16;
    if (n >= a.n) return;
    float bias[16];
    if constexpr (MODE == kForward)
      if (a.has_bias)
        load16<T>(bias, static_cast<const S*>(a.bias.get(int(job.rank))) + (uint64_t(job.expert) * a.n + n), n, a.n);
    constexpr int V = 16 / int(sizeof(S)), B = MF < 4 ? MF : 4;
    // Large forward products: what a tile's epilogue reads and writes is
    // twice the L2 of all its XCD's tiles, and would drive the operands out
    // of it.  With nontemporal accesses 32,768 rows 2560 -> 5120 with bias,
    // SiLU and residual take 930 us instead of 990, and without an epilogue
    // 8 x 4,096 rows 1,045 to 1,155 TFLOP/s; the gradients lose 3 %.
    constexpr bool kStream = MODE == kForward && MF == 8;
#pragma unroll
    for (int i0 = 0; i0 < MF; i0 += B) {
      // the residuals of B rows at once, into registers that the fragments had
      typename VecOf<S, V>::type res[B][16 / V];
      if constexpr (MODE == kForward)
        if (a.has_residual) {
          const S* residual = static_cast<const S*>(a.residual.get(int(job.rank))) + uint64_t(job.lo) * a.n + n;
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const uint32_t m = job.m0 + uint32_t(wm) * MF * 16 + uint32_t(i0 + i) * 16 + l % 16;
            if (m < m_end(job))
#pragma unroll
              for (int u = 0; u < 16 / V; ++u)
                res[i][u] = cut<S, kStream>(residual + uint64_t(m) * a.n + u * V, n + uint32_t(u * V), a.n);
          }
        }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const uint32_t m = job.m0 + uint32_t(wm) * MF * 16 + uint32_t(i0 + i) * 16 + l % 16;
        if (m >= m_end(job)) continue;
        const uint64_t row = MODE == kGradWeights ? uint64_t(job.expert) * a.m + m : uint64_t(job.lo) + m;
        const uint64_t at = row * a.n + n;
        float v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) v[j * 4 + u] = acc[i0 + i][j][u];
        if constexpr (MODE == kForward) {
          if (a.has_bias)
#pragma unroll
            for (int u = 0; u < 16; ++u) v[u] += bias[u];
          if (a.has_preact) store16<T, kStream>(static_cast<S*>(const_cast<void*>(a.preact.get(int(job.rank)))) + at, v, n, a.n);
          if (a.activation != CCL_SIM_ACT_NONE)
#pragma unroll
            for (int u = 0; u < 16; ++u) v[u] = activate<T>(v[u], a.activation);
          if (a.has_residual)
#pragma unroll
            for (int u = 0; u < 16; ++u) v[u] += T::widen(res[i][u / V][u % V]);
        }
        if (MODE == kGradWeights && a.splits > 1)
          store16<F32>(a.parts + (uint64_t(job.split) * a.nranks + job.rank) * a.per_rank * a.m * a.n + at, v, n, a.n);
        else
          store16<T, kStream>(static_cast<S*>(const_cast<void*>(a.out.get(int(job.rank)))) + at, v, n, a.n);
      }
    }
  };

  Job job = next_job();
  if (!job.on) return;
  enter(job);
  fetch(job, 0);
  settle();
  fetch(job, 1);
  Frags first, second;
  wait_all.template operator()<TA::kLoads + TB::kLoads>();
  uint32_t d = 0;  // stages multiplied so far; its parity names the buffer
  // The products of a stage, during which stage `s` of tile `j` is fetched.
  auto stage = [&](const Job& j, uint32_t s) {
    read(second, d, 1);
    products(first);
    settle();
    wait_all.template operator()<0>();
    fetch(j, s);
    ++d;
    read(first, d, 0);
    products(second);
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = float4_t{0, 0, 0, 0};
    read(first, d, 0);
    // At least two stages, so that the two fetched ahead reach no further
    // than the next tile; the last two run while that one's first two are
    // fetched (of no next tile: loads of nothing).  The fragments read ahead
    // in the very last are not kept, but read again after the epilogue,
    // which has the registers meanwhile and runs while loads are in flight.
    const uint32_t stages = (k_end(job) + El::kStage - 1) / El::kStage;
    for (uint32_t s = 2; s < stages; ++s) stage(job, s);
    const Job next = next_job();
    enter(next);
#pragma unroll 1
    for (uint32_t s = 0; s < 2; ++s) stage(next, s);
    store(job);
    if (!next.on) break;
    job = next;
  }
  // no load may still be writing to LDS when the workgroup gives it up
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---------------------------------------------------------------------------
// The forward product of few rows per expert (a serving step).  What bounds
// it is reading the weights of the experts that have rows, once, so nothing
// of them goes through LDS: a lane loads its 16 bytes of a fragment straight
// from memory, in the layout the matrix instruction wants, and what counts is
// how many such loads are in flight.  A workgroup takes 64 columns of one
// expert; its four waves take turns along k, 128 bytes each, so a wave's 8
// weight loads of a turn cover 64 whole lines, and the next turn's are
// started before the products of this one.  The waves' sums are added in
// LDS, in order, and wave j finishes the columns of fragment j.  An expert has
// at most the 16 rows of one fragment; those with more are left to the tiles.
// 8 experts of 8 rows, 2048 -> 2048:
// bf16 18 us (67 MB, 3.7 TB/s), float32 32 us (4.2 TB/s); 64 experts 2048 ->
// 4096 float32 (2.1 GB) 523 us, 4.1 TB/s.
// ---------------------------------------------------------------------------
constexpr uint32_t kFewRows = 16;

template <class T>
__global__ __launch_bounds__(256) void few_rows_kernel(ProductArgs a) {
  using S = typename T::S;
  using El = Elem<S>;
  using Chunk = typename VecOf<S, El::kChunk>::type;
  __shared__ float4_t part[4][4][kWave];
  const uint32_t block = blockIdx.x % a.ntiles, q = blockIdx.x / a.ntiles;
  const uint32_t rank = q / a.per_rank, expert = q - rank * a.per_rank;
  const int* off = a.has_offsets ? static_cast<const int*>(a.offsets.get(int(rank))) : nullptr;
  const Range r = rows_of(off, expert, a.capacity);
  const uint32_t lo = uniform(r.lo), rows = uniform(r.hi) - lo;
  if (rows == 0 || rows > kFewRows) return;
  const uint32_t l = uint32_t(lane_id()), i = l % 16, g = l / 16, w = uint32_t(wave_id());
  const uint32_t n0 = block * kWaveN;
  // this lane's weight rows (one per fragment) and its row, and their k within a half; past the last the last, not stored
  const S* wrow[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t n = n0 + 16 * (i / 4) + 4 * uint32_t(j) + i % 4;
    n = n < a.n ? n : a.n - 1;
    wrow[j] = static_cast<const S*>(a.b.get(int(rank))) + (uint64_t(expert) * a.n + n) * a.k + g * El::kChunk;
  }
  const S* xrow = static_cast<const S*>(a.a.get(int(rank))) + uint64_t(lo + (i < rows ? i : rows - 1)) * a.k + g * El::kChunk;
  float4_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = float4_t{0, 0, 0, 0};
  struct Turn {
    Chunk w[4][2], x[2];
  };
  // The loads of k from k0 on; `whole`: all of it inside k.
  auto load = [&](Turn& u, uint32_t k0, bool whole) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = k0 + uint32_t(h) * (El::kStage / 2);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u.w[j][h] = whole ? vload<S, El::kChunk, true>(wrow[j] + at) : cut(wrow[j] + at, at + g * El::kChunk, a.k);
      u.x[h] = whole ? vload<S, El::kChunk, false>(xrow + at) : cut(xrow + at, at + g * El::kChunk, a.k);
    }
  };
  auto products = [&](const Turn& u) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j] = multiply<T>(__builtin_bit_cast(float4_t, u.w[j][h]), __builtin_bit_cast(float4_t, u.x[h]), acc[j]);
  };
  constexpr uint32_t kTurn = 4 * El::kStage;
  uint32_t k0 = w * El::kStage;
  Turn now, next;
  if (k0 + El::kStage <= a.k) load(now, k0, true);
  for (; k0 + kTurn + El::kStage <= a.k; k0 += kTurn) {
    load(next, k0 + kTurn, true);
    products(now);
    now = next;
  }
  if (k0 + El::kStage <= a.k) {
    products(now);
    k0 += kTurn;
  }
  if (k0 < a.k) {
    load(now, k0, false);
    products(now);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) part[w][j][l] = acc[j];
  __syncthreads();
  const uint32_t n = n0 + g * 16 + w * 4;
  const float4_t sum = (part[0][w][l] + part[1][w][l]) + (part[2][w][l] + part[3][w][l]);
  if (i >= rows) return;
  const uint64_t at = uint64_t(lo + i) * a.n + n;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (n + u >= a.n) continue;
    float v = sum[u];
    if (a.has_bias) v += T::widen(get1(static_cast<const S*>(a.bias.get(int(rank))) + uint64_t(expert) * a.n + n + u));
    if (a.has_preact) put1(static_cast<S*>(const_cast<void*>(a.preact.get(int(rank)))) + at + u, round_to<T>(v));
    v = activate<T>(v, a.activation);
    if (a.has_residual) v += T::widen(get1(static_cast<const S*>(a.residual.get(int(rank))) + at + u));
    put1(static_cast<S*>(const_cast<void*>(a.out.get(int(rank)))) + at + u, round_to<T>(v));
  }
}

// ---------------------------------------------------------------------------
// The activation's gradient dz = g · act'(z), and its partial sums over
// `chunk` rows of one expert for the bias's gradient.  Memory-bound: g and z
// are read once, dz written once.  A workgroup takes a chunk of rows and the
// columns of 64 vectors, its waves every fourth row, four of them in flight.
// dz rows are `ldz` elements apart, zeros behind the last feature.
// ---------------------------------------------------------------------------
struct SlopeArgs {
  RankPtrs grads, preact, offsets;
  void* dz;
  float* sums;
  uint32_t per_rank, capacity, features, ldz, chunk, slots;
  uint32_t wide;  // workgroups across the columns
  bool has_offsets, want_sums;
  int activation;
};

template <class T>
__global__ __launch_bounds__(256) void slope_kernel(SlopeArgs a) {
  using S = typename T::S;
  constexpr int V = 16 / int(sizeof(S)), U = 4;
  using Vec = typename VecOf<S, V>::type;
  __shared__ float part[4][kWave * V];
  const uint32_t rank = blockIdx.y, slot = blockIdx.x / a.wide;
  const int* off = a.has_offsets ? static_cast<const int*>(a.offsets.get(int(rank))) : nullptr;
  const Range r = find_tile(off, a.per_rank, a.capacity, slot, a.chunk);
  if (r.expert >= a.per_rank) return;
  const uint32_t lo = r.lo + r.tile * a.chunk;
  const uint32_t hi = lo + a.chunk < r.hi ? lo + a.chunk : r.hi;
  const uint32_t l = uint32_t(lane_id()), w = uint32_t(wave_id());
  const uint32_t f = (blockIdx.x % a.wide * kWave + l) * V;
  const bool act = a.activation != CCL_SIM_ACT_NONE;
  const S* g = static_cast<const S*>(a.grads.get(int(rank))) + f;
  const S* z = act ? static_cast<const S*>(a.preact.get(int(rank))) + f : nullptr;
  S* dz = static_cast<S*>(a.dz) + uint64_t(rank) * a.capacity * a.ldz + f;
  float sum[V] = {};
  for (uint32_t s0 = lo + w; s0 < hi; s0 += 4 * U) {
    Vec gv[U], zv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t s = s0 + 4 * uint32_t(u);
      gv[u] = zv[u] = Vec{};
      if (s >= hi) continue;
      gv[u] = cut<S>(g + uint64_t(s) * a.features, f, a.features);
      if (act) zv[u] = cut<S>(z + uint64_t(s) * a.features, f, a.features);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t s = s0 + 4 * uint32_t(u);
      if (s >= hi) continue;
      Vec out;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float d = T::widen(gv[u][i]);
        if (act) d *= slope<T>(T::widen(zv[u][i]), a.activation);
        sum[i] += d;
        // bf16: rounded here, once, so that the two products take it as a
        // matrix operand; a relative error of at most 2^-8 per term, like
        // the rounding of the result
        out[i] = round_to<T>(d);
      }
      // dz is g itself without an activation; `ldz` is whole vectors when it
      // is not `features`, so the vector that holds the end fits its row
      if (!act || f >= a.ldz) continue;
      if (f + V <= a.ldz) {
        vstore<S, V, false>(dz + uint64_t(s) * a.ldz, out);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (f + uint32_t(i) < a.ldz) put1(dz + uint64_t(s) * a.ldz + i, out[i]);
      }
    }
  }
  if (!a.want_sums) return;
#pragma unroll
  for (int i = 0; i < V; ++i) part[w][i * kWave + l] = sum[i];
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (f + i < a.features) {
        const float t = (part[0][i * kWave + l] + part[1][i * kWave + l]) + (part[2][i * kWave + l] + part[3][i * kWave + l]);
        put1(a.sums + (uint64_t(rank) * a.slots + slot) * a.features + f + i, t);
      }
  }
}

// The bias's gradient: the sum of an expert's partial sums.  A workgroup
// takes 64 columns of an expert, its 8 waves every eighth slot, in order.
struct BiasArgs {
  RankPtrs offsets, grad_bias;
  const float* sums;
  uint32_t per_rank, capacity, features, chunk, slots;
  bool has_offsets;
};

template <class T>
__global__ __launch_bounds__(512) void bias_kernel(BiasArgs a) {
  using S = typename T::S;
  constexpr int W = 8, U = 8;
  __shared__ float part[W][kWave];
  const uint32_t rank = blockIdx.z, expert = blockIdx.y;
  const uint32_t l = uint32_t(lane_id()), w = uint32_t(wave_id()), f = blockIdx.x * kWave + l;
  const int* off = a.has_offsets ? static_cast<const int*>(a.offsets.get(int(rank))) : nullptr;
  auto slots_of = [&](uint32_t e) {
    const Range r = rows_of(off, e, a.capacity);
    return (r.hi - r.lo + a.chunk - 1) / a.chunk;
  };
  uint32_t first = 0;
  for (uint32_t e = l; e < expert; e += kWave) first += slots_of(e);
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) first += uint32_t(__shfl_xor(int(first), d));
  uint32_t end = first + slots_of(expert);
  end = end < a.slots ? end : a.slots;  // only offsets that overlap reach past the slots
  const float* sums = a.sums + uint64_t(rank) * a.slots * a.features + f;
  float sum = 0.0f;
  for (uint32_t s0 = first + w; s0 < end; s0 += W * U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t s = s0 + W * uint32_t(u);
      v[u] = f < a.features && s < end ? get1(sums + uint64_t(s) * a.features) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) sum += v[u];
  }
  part[w][l] = sum;
  __syncthreads();
  if (w != 0 || f >= a.features) return;
  float total = 0.0f;
#pragma unroll
  for (int u = 0; u < W; ++u) total += part[u][l];
  put1(static_cast<S*>(const_cast<void*>(a.grad_bias.get(int(rank)))) + uint64_t(expert) * a.features + f, round_to<T>(total));
}

// ---------------------------------------------------------------------------
// A copy of a matrix's rows with a stride of whole 16-byte vectors, zeros
// behind each row's end: rows that do not start on 16 bytes cannot be loaded
// straight to LDS.  A wave per row; where the rows are the experts' tokens,
// only those up to the largest of the rank's offsets.
// ---------------------------------------------------------------------------
struct PackArgs {
  RankPtrs in, offsets;
  void* out;
  uint32_t rows, per_rank, width, ld;  // rows of a rank; elements of a row; the copy's stride
  bool ragged;
};

template <class S>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a) {
  constexpr int V = 16 / int(sizeof(S)), U = 4;
  const uint32_t rank = blockIdx.y;
  uint32_t rows = a.rows;
  if (a.ragged) {
    // the last offset, unless offsets decrease: an expert before may end later
    const int* off = static_cast<const int*>(a.offsets.get(int(rank)));
    rows = 0;
    for (uint32_t e = uint32_t(lane_id()); e <= a.per_rank; e += kWave) {
      const uint32_t v = offset_at(off, e, a.rows);
      rows = v > rows ? v : rows;
    }
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2) {
      const uint32_t v = uint32_t(__shfl_xor(int(rows), d));
      rows = v > rows ? v : rows;
    }
    rows = uniform(rows);
  }
  const S* in = static_cast<const S*>(a.in.get(int(rank)));
  S* out = static_cast<S*>(a.out) + uint64_t(rank) * a.rows * a.ld;
  for (uint32_t r = blockIdx.x * 4 + uint32_t(wave_id()); r < rows; r += gridDim.x * 4) {
    for (uint32_t i0 = uint32_t(lane_id()) * V; i0 < a.ld; i0 += kWave * V * U) {
      typename VecOf<S, V>::type v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + uint32_t(u) * kWave * V;
        if (i < a.ld) v[u] = cut<S>(in + uint64_t(r) * a.width + i, i, a.width);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + uint32_t(u) * kWave * V;
        if (i < a.ld) vstore<S, V, false>(out + uint64_t(r) * a.ld + i, v[u]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The weights' gradient as the sum of `splits` float32 parts, in order.
// ---------------------------------------------------------------------------
struct JoinArgs {
  RankPtrs out;
  const float* parts;  // [splits][nranks][count]
  uint64_t count;      // elements of a rank
  uint32_t nranks, splits;
};

template <class T>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a) {
  using S = typename T::S;
  constexpr int V = 16 / int(sizeof(S));
  const uint32_t rank = blockIdx.y;
  S* out = static_cast<S*>(const_cast<void*>(a.out.get(int(rank))));
  const float* in = a.parts + uint64_t(rank) * a.count;
  for (uint64_t i = (uint64_t(blockIdx.x) * 256 + threadIdx.x) * V; i < a.count; i += uint64_t(gridDim.x) * 256 * V) {
    float sum[V] = {};
    const bool whole = i + V <= a.count;
    for (uint32_t p = 0; p < a.splits; ++p) {
      const float* q = in + uint64_t(p) * a.nranks * a.count + i;
      if (whole) {
        const auto v = vload<float, V, false>(q);
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] += v[k];
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (i + uint64_t(k) < a.count) sum[k] += get1(q + k);
      }
    }
    typename VecOf<S, V>::type o;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = round_to<T>(sum[k]);
    if (whole) {
      vstore<S, V, false>(out + i, o);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (i + uint64_t(k) < a.count) put1(out + i + k, o[k]);
    }
  }
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------
// An operand as the launches see it: the caller's buffers, or a copy in the
// workspace.
struct Operand {
  const RankPtrs* ranks = nullptr;
  bool aligned = false;        // every rank's buffer starts on 16 bytes
  const char* at = nullptr;    // the copy, its ranks `step` bytes apart
  uint64_t step = 0;
  uint32_t ld = 0;
};

// A launch holds fewer than 2^32 threads, of which a workgroup has up to 512.
constexpr uint64_t kMostBlocks = uint64_t(1) << 22;

template <class T, int MODE>
hipError_t launch_product(const ProductCall& c, ProductArgs a, const Operand& x, const Operand& y) {
  using S = typename T::S;
  const uint32_t size = sizeof(S);
  a.a = *x.ranks;
  a.b = *y.ranks;
  a.a_at = x.at;
  a.b_at = y.at;
  a.a_step = x.step;
  a.b_step = y.step;
  a.lda = x.ld;
  a.ldb = y.ld;
  if (a.splits == 0) a.splits = 1;
  // the loads to LDS move 16 bytes: rows and base addresses start on that
  const bool direct = x.aligned && y.aligned && x.ld * size % 16 == 0 && y.ld * size % 16 == 0;
  auto go = [&](auto kernel, uint32_t bm, uint32_t bn, uint32_t threads, uint32_t per_cu) -> hipError_t {
    a.ntiles = (a.n + bn - 1) / bn;
    uint64_t grid;
    if (MODE == kGradWeights) {
      const uint64_t tiles = uint64_t((a.m + bm - 1) / bm) * a.ntiles;
      grid = uint64_t(a.nranks) * a.per_rank * a.splits * ((tiles + 7) / 8) * 8;
      if (grid > kMostBlocks) grid = kMostBlocks;
    } else {
      // as many workgroups as run at once, or as there may be tiles
      const uint64_t mtiles = a.has_offsets ? a.capacity / bm + a.per_rank : (a.capacity + bm - 1) / bm;
      const uint64_t most = (uint64_t(a.nranks) * mtiles * a.ntiles + 7) / 8 * 8;
      grid = uint64_t(c.num_cus) * per_cu / 8 * 8;
      if (grid < 8) grid = 8;
      if (most < grid) grid = most;
    }
    if (grid == 0) return hipSuccess;
    if (c.log_plan)
      std::fprintf(stderr, "[ccl_sim] product %s %s: tiles of %u x %u by %u threads, loads %s, %llu workgroups\n",
                   MODE == kForward ? "forward" : MODE == kGradRows ? "grad_rows" : "grad_weights",
                   size == 2 ? "bf16" : "float32", bm, bn, threads, direct ? "to LDS" : "by registers",
                   static_cast<unsigned long long>(grid));
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(threads), 0, c.stream, a);
    return hipGetLastError();
  };
  // The tile: the largest that gives every compute unit at least one.  What
  // a smaller tile costs is its operands' way from the L2 to LDS, which a
  // 256 x 256 tile takes half as often as a 128 x 128 one; what too few
  // tiles cost is idle compute units.  The rows are taken as spread evenly
  // over a full capacity, which is all that the host knows of them.
  auto tiles = [&](uint64_t bm, uint64_t bn) {
    const uint64_t wide = (a.n + bn - 1) / bn, experts = uint64_t(a.nranks) * a.per_rank;
    if (MODE == kGradWeights) return experts * a.splits * ((a.m + bm - 1) / bm) * wide;
    return experts * ((a.capacity / a.per_rank + bm - 1) / bm) * wide;
  };
  const uint64_t cus = uint64_t(c.num_cus);
  if (!direct) {
    // Rows off the 16-byte grid, loaded through registers: what counts is
    // having other waves to run while a stage's loads arrive, so 8 waves
    // share a tile (460 rows, rows' gradient of 4095 -> 4097 bf16: 180 us, 257 with 4).
    if (tiles(64, 128) * 4 >= cus * 3) return go(product_kernel<T, MODE, false, 1, 4, 2>, 64, 128, 512, 2);
    return go(product_kernel<T, MODE, false, 1, 4, 1>, 64, 64, 256, 4);
  }
  // (experts of few rows would leave most of a tall tile empty)
  const uint64_t each = MODE == kGradWeights ? a.m : a.capacity / a.per_rank;
  if constexpr (sizeof(S) == 2)
    if (each > 128 && tiles(256, 256) >= cus) return go(product_kernel<T, MODE, true, 8, 2, 4>, 256, 256, 512, 1);
  if constexpr (sizeof(S) == 2) {
    // Between a quarter and three quarters more or less than one tile per
    // compute unit, measured (us, tiles of 128 x 128 / 64 x 128 / 64 x 64):
    // 1,850 rows 2048 -> 2048 (240 / 480 / 960 tiles) 28.9 / 26.3 / -; 9
    // experts of 330 rows 1736 -> 1000 (216 / 432 / 864) 30.1 / 28.8 / 41.3,
    // 1000 -> 1736 (378 / 756 / 1,512) 28.1 / 32.5 / -; 920 rows 2048 -> 2048
    // (128 / 240 / 480) 24.4 / 21.9 / 26.1.
    if (each > 64 && tiles(128, 128) * 4 >= cus * 5) return go(product_kernel<T, MODE, true, 4, 2, 2>, 128, 128, 256, 2);
    if (tiles(64, 128) * 4 >= cus * 3) return go(product_kernel<T, MODE, true, 2, 2, 2>, 64, 128, 256, 3);
  } else {
    // the matrix units bound at either tile: 64 x 64 and 128 x 128 are equal
    // where both fill the GPU, and 128 x 128 takes twice as long at half of it
    if (each > 64 && tiles(128, 128) >= cus) return go(product_kernel<T, MODE, true, 4, 2, 2>, 128, 128, 256, 2);
  }
  return go(product_kernel<T, MODE, true, 1, 4, 1>, 64, 64, 256, 4);
}

ProductArgs product_args(const ProductCall& c) {
  ProductArgs a{};
  a.offsets = c.offsets;
  a.nranks = uint32_t(c.nranks);
  a.per_rank = c.per_rank;
  a.capacity = c.capacity;
  a.has_offsets = c.has_offsets;
  a.activation = CCL_SIM_ACT_NONE;
  return a;
}

// `x`, its rows copied to `at` with stride `ld`; `rows` of a rank, `ragged`
// where they are the experts' tokens.
template <class S>
hipError_t pack(const ProductCall& c, Operand& x, size_t at, uint32_t rows, uint32_t width, uint32_t ld, bool ragged) {
  PackArgs p{};
  p.in = *x.ranks;
  p.offsets = c.offsets;
  p.out = c.scratch + at;
  p.rows = rows;
  p.per_rank = c.per_rank;
  p.width = width;
  p.ld = ld;
  p.ragged = ragged && c.has_offsets;
  x.at = c.scratch + at;
  x.step = uint64_t(rows) * ld * sizeof(S);
  x.ld = ld;
  x.aligned = true;
  const uint32_t blocks = (rows + 3) / 4, most = 4096;
  hipLaunchKernelGGL(pack_kernel<S>, dim3(blocks < most ? blocks : most, unsigned(c.nranks)), dim3(256), 0, c.stream, p);
  return hipGetLastError();
}

ProductPlan plan_of(const ProductCall& c) {
  return product_plan(c.dtype, uint32_t(c.nranks), c.per_rank, c.capacity, c.hidden, c.features);
}

template <class T>
hipError_t matmul(const ProductCall& c) {
  using S = typename T::S;
  ProductArgs a = product_args(c);
  a.out = c.out;
  a.bias = c.bias;
  a.residual = c.residual;
  a.preact = c.preact;
  a.n = c.features;
  a.k = c.hidden;
  a.has_bias = c.has_bias;
  a.has_residual = c.has_residual;
  a.has_preact = c.has_preact;
  a.activation = c.activation;
  const uint32_t rows = c.capacity / c.per_rank;
  // The form for few rows: up to one pass of 16 rows over the weights per expert
  // on average, where its workgroups (64 columns of an expert each) are no more
  // than the compute units; of float32 with rows on the 16-byte grid also where
  // they are no more than twice that, or hidden is at most 2048, so that the
  // tiles have few stages.  Measured (us, tiles / few rows; weights from memory
  // and, in brackets, from the caches):
  //   workgroups, bf16, 8 rows an expert: 64 (2048 -> 4096) 30 / 15 [17 / 13],
  //     128 19 / 10 [13 / 10], 256 (2048 -> 2048) 32 / 18 [23 / 17], 256 (5120 ->
  //     4096) 66 / 43 [45 / 42]; 320 34 / 29 [23 / 28], 512 40 / 35 [27 / 33],
  //     1,024 30 / 33 [26 / 32], 2,560 138 / 158, 5120 -> 2560 with 1,280 160 / 205;
  //     of odd widths 65 (4097 -> 4097) 68 / 64 [52 / 64], 256 40 / 30 [31 / 29],
  //     512 49 / 54; in between it is by the shape: 2048 -> 4096 with 2,048 127 /
  //     120, 32 rows over those 32 experts at random 77 / 70
  //   float32: 256 58 / 32 [49 / 31], 512 82 / 66 (8192 -> 4096 286 / 247), 1,024
  //     87 / 70, 4,096 289 / 254; 4096 -> 2048 with 1,024 274 / 278, 5120 -> 2560
  //     with 1,280 412 / 453; of odd widths 256 66 / 42, 512 91 / 88, 1,024 85 / 93
  //   rows an expert, 256 workgroups, bf16: 16 32 / 19 [23 / 18], 32 32 / 34 [23 / 33];
  //     float32: 16 58 / 33 [49 / 33], 32 58 / 64 [49 / 64]
  const uint32_t columns = (a.n + kWaveN - 1) / kWaveN;
  const uint64_t blocks = uint64_t(a.nranks) * a.per_rank * columns, cus = uint64_t(c.num_cus);
  const bool wide = sizeof(S) == 4 && c.rows16 && c.weights16 && c.hidden * sizeof(S) % 16 == 0 &&
                    (blocks <= 2 * cus || c.hidden <= 2048);
  if (rows <= kFewRows && (blocks <= cus || wide)) {
    // An expert may still have more: those are left to the tiles, in a second
    // launch where the capacity allows for any (2.5 us when there are none).
    if (c.capacity > kFewRows && c.has_offsets) a.least = kFewRows + 1;
    ProductArgs few = a;
    few.a = c.rows;
    few.b = c.weights;
    few.ntiles = columns;
    const dim3 grid(a.nranks * a.per_rank * few.ntiles);
    if (c.log_plan)
      std::fprintf(stderr, "[ccl_sim] product forward %s: few rows, %u workgroups\n", sizeof(S) == 2 ? "bf16" : "float32", grid.x);
    hipLaunchKernelGGL(few_rows_kernel<T>, grid, dim3(256), 0, c.stream, few);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.least == 0) return e;
  }
  const ProductPlan plan = plan_of(c);
  Operand x{&c.rows, c.rows16, nullptr, 0, c.hidden}, w{&c.weights, c.weights16, nullptr, 0, c.hidden};
  if (plan.pack_hidden) {
    hipError_t e = pack<S>(c, x, plan.rows, c.capacity, c.hidden, plan.ldh, true);
    if (e == hipSuccess) e = pack<S>(c, w, plan.weights, c.per_rank * c.features, c.hidden, plan.ldh, false);
    if (e != hipSuccess) return e;
  }
  return launch_product<T, kForward>(c, a, x, w);
}

template <class T>
hipError_t matmul_grad(const ProductCall& c) {
  using S = typename T::S;
  constexpr uint32_t V = 16 / sizeof(S);
  hipError_t e = hipSuccess;
  const bool act = c.activation != CCL_SIM_ACT_NONE;
  const ProductPlan plan = plan_of(c);
  if ((act || c.want_bias) && c.capacity > 0 && c.features > 0) {
    SlopeArgs s{};
    s.grads = c.grads;
    s.preact = c.preact;
    s.offsets = c.offsets;
    s.dz = c.scratch + plan.dz;
    s.sums = reinterpret_cast<float*>(c.scratch + plan.sums);
    s.per_rank = c.per_rank;
    s.capacity = c.capacity;
    s.features = c.features;
    s.ldz = plan.ldf;
    s.chunk = plan.chunk;
    s.slots = plan.slots;
    s.has_offsets = c.has_offsets;
    s.want_sums = c.want_bias;
    s.activation = c.activation;
    s.wide = (c.features + kWave * V - 1) / (kWave * V);
    hipLaunchKernelGGL(slope_kernel<T>, dim3(s.wide * s.slots, unsigned(c.nranks)), dim3(256), 0, c.stream, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (c.want_bias && c.features > 0) {
    BiasArgs b{};
    b.offsets = c.offsets;
    b.grad_bias = c.grad_bias;
    b.sums = reinterpret_cast<const float*>(c.scratch + plan.sums);
    b.per_rank = c.per_rank;
    b.capacity = c.capacity;
    b.features = c.features;
    b.chunk = plan.chunk;
    b.slots = plan.slots;
    b.has_offsets = c.has_offsets;
    hipLaunchKernelGGL(bias_kernel<T>, dim3((c.features + kWave - 1) / kWave, c.per_rank, unsigned(c.nranks)), dim3(512),
                       0, c.stream, b);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  Operand dz{&c.grads, c.grads16, nullptr, 0, c.features};
  if (act) {
    dz = Operand{&c.grads, true, c.scratch + plan.dz, uint64_t(c.capacity) * plan.ldf * sizeof(S), plan.ldf};
  } else if (plan.pack_features && c.capacity > 0 && (c.want_rows || c.want_weights)) {
    e = pack<S>(c, dz, plan.dz, c.capacity, c.features, plan.ldf, true);
    if (e != hipSuccess) return e;
  }
  if (c.want_rows) {
    ProductArgs a = product_args(c);
    Operand w{&c.weights, c.weights16, nullptr, 0, c.hidden};
    if (plan.pack_hidden) {
      e = pack<S>(c, w, plan.grad_weights, c.per_rank * c.features, c.hidden, plan.ldh, false);
      if (e != hipSuccess) return e;
    }
    a.out = c.grad_rows;
    a.n = c.hidden;
    a.k = c.features;
    e = launch_product<T, kGradRows>(c, a, dz, w);
    if (e != hipSuccess) return e;
  }
  if (c.want_weights && c.features > 0) {
    ProductArgs a = product_args(c);
    Operand x{&c.rows, c.rows16, nullptr, 0, c.hidden};
    if (plan.pack_hidden) {
      e = pack<S>(c, x, plan.grad_rows, c.capacity, c.hidden, plan.ldh, true);
      if (e != hipSuccess) return e;
    }
    a.out = c.grad_weights;
    a.m = c.features;
    a.n = c.hidden;
    a.splits = plan.splits;
    a.parts = reinterpret_cast<float*>(c.scratch + plan.parts);
    e = launch_product<T, kGradWeights>(c, a, dz, x);
    if (e != hipSuccess || plan.splits == 1) return e;
    JoinArgs j{};
    j.out = c.grad_weights;
    j.parts = a.parts;
    j.count = uint64_t(c.per_rank) * c.features * c.hidden;
    j.nranks = uint32_t(c.nranks);
    j.splits = plan.splits;
    const uint64_t blocks = (j.count + 256 * V - 1) / (256 * V);
    hipLaunchKernelGGL(join_kernel<T>, dim3(unsigned(blocks < 4096 ? blocks : 4096), unsigned(c.nranks)), dim3(256), 0,
                       c.stream, j);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

// Copies pay when the product's time saved by loads straight to LDS (about
// half of its time) is more than that of reading and writing the operands
// once more and two launches.  Measured on bf16 of odd widths, against the
// register path: 8 ranks of 4,096 rows, 2047 -> 4095, forward 1,263 to
// 619 us, rows' gradient 2,176 to 599, weights' 1,763 to 561; 3,300 rows over
// 9 experts, 1001 -> 1735, which the rule leaves alone, takes 47 us, 26 with
// even widths, and the copies would be 76 MB.
//
// Splits: an expert's weights' gradient sums over its rows, and there are few
// 128 x 128 tiles of it when the matrix is small; then the rows are cut so
// that the 256 compute units of the GPU get a tile each and some, of 512 rows
// or more (16,384 rows of 512 x 512 bf16: 103 us without, 31 with 16 or 20).
ProductPlan product_plan(int dtype, uint32_t nranks, uint32_t per_rank, uint32_t capacity, uint32_t hidden,
                         uint32_t features) {
  ProductPlan p;
  const uint64_t es = elem_size(dtype), v = 16 / es;
  const uint64_t rows = uint64_t(nranks) * capacity, experts = uint64_t(nranks) * per_rank;
  const uint64_t h = hidden, f = features;
  const bool pays = rows * f / 256 * h > rows * h + experts * f * h + (uint64_t(4) << 20);
  p.pack_hidden = pays && h % v != 0;
  p.pack_features = pays && f % v != 0;
  p.ldh = uint32_t(p.pack_hidden ? (h + v - 1) / v * v : h);
  p.ldf = uint32_t(p.pack_features ? (f + v - 1) / v * v : f);
  const uint64_t tiles = experts * ((f + 127) / 128) * ((h + 127) / 128), each = capacity / per_rank;
  if (tiles > 0 && tiles < 256) {
    const uint64_t want = (320 + tiles - 1) / tiles, most = each / 512;
    p.splits = uint32_t(want < most ? want : most);
    if (p.splits < 1) p.splits = 1;
  }
  const uint64_t wide = (f + 64 * v - 1) / (64 * v);
  p.chunk = 16;
  while (p.chunk < 512 && rows / p.chunk * wide > 4096) p.chunk *= 2;
  p.slots = capacity / p.chunk + per_rank;

  auto part = [](size_t& off, uint64_t bytes) {
    const size_t at = off;
    off += size_t((bytes + 255) / 256 * 256);
    return at;
  };
  p.rows = part(p.forward, p.pack_hidden ? rows * p.ldh * es : 0);
  p.weights = part(p.forward, p.pack_hidden ? experts * f * p.ldh * es : 0);
  p.dz = part(p.grads, rows * p.ldf * es);
  p.sums = part(p.grads, uint64_t(nranks) * p.slots * f * 4);
  p.parts = part(p.grads, p.splits > 1 ? p.splits * experts * f * h * 4 : 0);
  p.grad_rows = part(p.grads, p.pack_hidden ? rows * p.ldh * es : 0);
  p.grad_weights = part(p.grads, p.pack_hidden ? experts * f * p.ldh * es : 0);
  return p;
}

hipError_t run_expert_matmul(const ProductCall& c) {
  return c.dtype == kBFloat16 ? matmul<BF16>(c) : matmul<F32>(c);
}

hipError_t run_expert_matmul_grad(const ProductCall& c) {
  return c.dtype == kBFloat16 ? matmul_grad<BF16>(c) : matmul_grad<F32>(c);
}

}  // namespace ccl
