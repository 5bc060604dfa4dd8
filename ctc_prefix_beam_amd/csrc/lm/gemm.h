// The matrix product behind the token loss and its gradients:
//   C[m, n] = sum_k A(m, k) B(n, k),   float32 sums (of int8 operands int32, exact),
// with what follows the product done on the sums in registers (the Epilogue).
// Either operand may be stored with k contiguous (row m: k = 0..) or with m
// contiguous (row k: m = 0..), so that the products of the gradients read x, w
// and d as they are, without transposed copies.
//
// A workgroup computes BM x BN from tiles of 128 bytes of k per row (128 8-bit values, 64
// 16-bit ones or 32 floats), double-buffered in LDS and filled by loads that go
// straight there, 1 KB per wave instruction.  Such a load writes its 64 pieces
// of 16 bytes one after another, so the layout that spreads LDS reads over all
// banks is made by choosing which piece each lane fetches:
//   k contiguous: piece p of row r is at r*128 + (p ^ ((r >> 1) & 7)) * 16, so
//     that the 16 rows that a 16-byte fragment read touches fill all 256 bytes
//     of the banks once;
//   m contiguous: piece p of k-row k is at k*RB + (p ^ swizzle(k)) * 16, so that
//     the k-rows a fragment read touches lie in different banks.
// Pieces outside the operand are fetched as zeros (an offset past the buffer
// descriptor's range), so sizes need not be multiples of the tile.
#pragma once
#include "common.h"

namespace ctcpb_lm {

constexpr uint32_t kOutside = 0x80000000u;   // beyond every buffer descriptor's range

typedef __attribute__((address_space(3))) char lds_char;

template <typename T>
struct Frag;

template <>
struct Frag<__bf16> {
  typedef bf16x8 V;
  typedef f32x4 Sum;
  static constexpr int kMfma = 32;   // k of one fragment (over the four lane groups)
  static __device__ f32x4 mac(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<_Float16> {
  typedef f16x8 V;
  typedef f32x4 Sum;
  static constexpr int kMfma = 32;
  static __device__ f32x4 mac(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<float> {
  typedef f32x4 V;
  typedef f32x4 Sum;
  static constexpr int kMfma = 16;
  static __device__ f32x4 mac(V a, V b, f32x4 c) {
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
};

template <>
struct Frag<int8_t> {
  typedef i32x4 V;
  typedef i32x4 Sum;   // exact
  static constexpr int kMfma = 64;
  static __device__ i32x4 mac(V a, V b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};

// One operand: `rows` along m (or n) and K along k, element (m, k) at
// data[m*ld + k] (k contiguous) or data[k*ld + m] (m contiguous); ld in bytes,
// a multiple of 16, data 16-byte aligned.  Where m is contiguous, every row of
// the operand can be read up to the next multiple of 16 bytes.
// With `twice` (m contiguous only), rows k = 2i and 2i + 1 are both row i of the data.
struct Operand {
  const char* data;
  int64_t ld;
  int32_t rows;
  bool twice;
};

// A fetch straight into LDS: lane l's BYTES (4 or 16) from base + offset to lds +
// l*BYTES (zeros for offsets outside).  Written as assembly, with no register
// result, because the compiler makes every transposing LDS read wait for all fetches
// it knows of; the waits that are needed are those of wait_and_meet().
template <int BYTES>
__device__ inline void fetch_to_lds(const void* base, void* lds, uint32_t offset) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const u32x4 rsrc = {(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
  const uint32_t to = (uint32_t)(uintptr_t)(lds_char*)lds;
  // nothing else in these kernels uses m0 (the warning is about reserved registers)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(offset), "s"(rsrc)
                 : "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(offset), "s"(rsrc)
                 : "m0");
#pragma clang diagnostic pop
}

// N (a multiple of 64) floats from `from` on to `lds`, zeros past `count` of them,
// the fetches dealt to the W waves from wave `first` on.
template <int N, int W>
__device__ inline void fetch_floats(const void* from, int count, float* lds, int first, int wave,
                                    int lane) {
#pragma unroll
  for (int i = 0; i < N / 64; ++i)
    if ((i + first) % W == wave) {
      const int k = i * 64 + lane;
      fetch_to_lds<4>(from, lds + i * 64, k < count ? (uint32_t)k * 4 : kOutside);
    }
}

// Fetches an R-row tile of an operand into LDS and reads fragments from it.
// W: waves of the workgroup.
template <typename T, int R, bool KC, int W>
struct TileLoader {
  static constexpr int kBK = 128 / sizeof(T);
  static constexpr int kPer = 16 / sizeof(T);     // elements of a piece
  static constexpr int kLoads = R / 8 / W;        // 1 KB loads per wave
  static constexpr int kRow = KC ? 128 : R * (int)sizeof(T);   // bytes of a row in LDS
  static constexpr int kPieces = kRow / 16;
  static constexpr int kReads = KC ? 1 : sizeof(T) == 2 ? 2 : 4;   // LDS reads of a fragment
  static_assert(R >= 64 && kLoads * 8 * W == R, "tile and waves do not match");
  typedef typename Frag<T>::V V;

  // A load covers kRows rows of the tile in LDS; its first row is wave-uniform, so a
  // lane keeps only its row and byte in the first load and derives the others.
  static constexpr int kRows = 64 / kPieces;

  const char* base;        // the next tile
  int64_t ld, step;        // bytes from row to row, from tile to tile
  int32_t lane_row;
  uint32_t lane_byte, lane_off;
  int32_t rows;            // rows (k contiguous) or bytes (m contiguous) left of m
  int32_t twice;

  // Row r of the tile has its piece p at p ^ swizzle(r): bits of r, so that
  // swizzle(a + b) = swizzle(a) ^ swizzle(b) where a and b share none.
  static __device__ int swizzle(int r) {
    if constexpr (KC)
      return (r >> 1) & 7;
    else if constexpr (sizeof(T) == 2 && R >= 128)
      return ((r & 3) | ((r >> 3) & 1) << 2) << 1;
    else if constexpr (sizeof(T) == 2)   // rows of 128 bytes, two to all the banks
      return (((r >> 1) & 1) | ((r >> 3) & 1) << 1) << 1;
    else
      return ((r >> 2) & 3) << 2;
  }

  __device__ void init(const Operand& o, int row0, int k0, int lane) {
    ld = o.ld;
    if constexpr (KC) {
      base = o.data + row0 * o.ld + (int64_t)k0 * (int)sizeof(T);
      step = 128;
      rows = o.rows - row0;
    } else {
      twice = o.twice ? 1 : 0;
      base = o.data + (k0 >> twice) * o.ld + (int64_t)row0 * (int)sizeof(T);
      step = (kBK >> twice) * o.ld;
      rows = min(o.rows - row0, R) * (int)sizeof(T);
    }
    lane_row = lane / kPieces;
    lane_byte = (lane % kPieces ^ swizzle(lane_row)) * 16;
    lane_off = (uint32_t)((KC ? lane_row : lane_row >> twice) * o.ld);
  }

  // Starts fetch q of the tile that begins `left` values of k before the operand's
  // end (0 or less: all zeros).
  __device__ void fetch(char* lds, int q, int left, int wave) const {
    const int first = (wave * kLoads + q) * kRows;
    const uint32_t byte = lane_byte ^ (uint32_t)(swizzle(first) * 16);
    const int row_end = (KC ? rows : left) - first;
    const int byte_end = KC ? min(left, kBK) * (int)sizeof(T) : rows;
    const uint32_t o = lane_row < row_end && (int)byte < byte_end ? lane_off + byte : kOutside;
    fetch_to_lds<16>(base + (KC ? first : first >> twice) * ld, lds + (wave * kLoads + q) * 1024, o);
  }

  // The whole tile; `base` moves on to the next one.
  __device__ void load(char* lds, int left, int wave) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) fetch(lds, q, left, wave);
    base += step;
  }

  // The fragment of rows r0 .. r0+15 (r0 a multiple of 16) and k-step kk.
  static __device__ V read(const char* lds, int r0, int kk, int lane) {
    const int g = lane >> 4, c = lane & 15;
    if constexpr (KC) {
      const int p = (kk * 4 + g) ^ swizzle(c);
      return *reinterpret_cast<const V*>(lds + (r0 + c) * 128 + p * 16);
    } else if constexpr (sizeof(T) == 2) {
      // two transposing reads of four k each: lane i of a group gives the address of
      // four values of k-row i/4 and receives the four k of column i
      typedef short s4 __attribute__((ext_vector_type(4)));
      const int k = kk * 32 + g * 8 + (c >> 2);
      const int p = (r0 / 8 + ((c & 3) >> 1)) ^ swizzle(g * 8 + (c >> 2));
      const char* at = lds + k * kRow + p * 16 + (c & 1) * 8;
      typedef __attribute__((address_space(3))) s4* ptr;
      const s4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char*)at);
      const s4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char*)(at + 4 * kRow));
      return __builtin_bit_cast(V, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      V v;
      const int p = (r0 / 4 + (c >> 2)) ^ swizzle(g * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const float*>(lds + (kk * 16 + g * 4 + j) * kRow + p * 16 +
                                               (c & 3) * 4);
      return v;
    }
  }
};

struct GemmArgs {
  Operand a, b;
  int32_t K;
  int32_t tiles_m, tiles_n;
  int32_t splits, part;   // parts of k, and the length of one (a multiple of the k-tile)
  int32_t n0;             // the epilogue's n of b's first row
};

// Where work item `id` lies.  Consecutive ids go to the eight XCDs in turn, so
// each XCD is given a contiguous range of the items, walked eight n-tiles wide,
// to find its operands in its own L2.
struct Place {
  int32_t m, n, split;   // tiles
  int32_t n0;            // the epilogue's n of the tile's first row
};
__device__ inline Place place_of(const GemmArgs& a, int id) {
  const int tiles = a.tiles_m * a.tiles_n, per = tiles * a.splits / 8;
  if (id < per * 8) id = (id % 8) * per + id / 8;
  Place p;
  p.split = id / tiles;
  id -= p.split * tiles;
  const int band = 8 * a.tiles_m;
  const int first = id / band * 8;
  const int wide = min(8, a.tiles_n - first);
  p.n = first + id % band % wide;
  p.m = id % band / wide;
  return p;
}

// Waits for this wave's fetches into LDS and its LDS reads, then for the other waves.
__device__ inline void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The order of the instructions behind it: `reads` LDS reads spread evenly over
// the first matrix instructions of `macs`; those after them hide the reads' latency.
template <int reads, int macs>
__device__ inline void interleave() {
  constexpr int span = macs > 8 ? macs - 8 : macs;
#pragma unroll
  for (int i = 0; i < macs; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a matrix instruction
    if (i < span) {
      const int n = reads * (i + 1) / span - reads * i / span;
      for (int r = 0; r < n; ++r) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
  }
}

// BM x BN per work item, WM x WN waves.  Workgroups stay for as many items as
// come to them: an item's first fetches are under way while the one before is
// finished by the epilogue.  LDS lets one, two or four workgroups of the three
// shapes share a CU; the registers have to leave room for them.
//
// Products of f32 are summed in parts of kPartTiles k-tiles.  One chain of K additions
// loses about sqrt(K) roundings of the whole sum, and the error of a logit is the
// relative error of its exponential: 3 x 319 x 1377 gradients 3.7e-6 off with one chain,
// under 1e-6 with parts.  The second set of sums does not fit beside that of a 256x256 tile,
// which f32 does not use for that reason (4096 x 16000 x 1024: loss 973 us with it
// and one chain, 1022 without).
template <typename T, int BM, int BN, int WM, int WN, bool AKC, bool BKC, typename Epilogue>
__global__ __launch_bounds__(64 * WM * WN, BM == 64 ? 4 : 2) void gemm_kernel(GemmArgs a, Epilogue ep) {
  constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  typedef TileLoader<T, BM, AKC, W> LA;
  typedef TileLoader<T, BN, BKC, W> LB;
  constexpr int kReads = TM * LA::kReads + TN * LB::kReads;
  constexpr int kMacs = TM * TN * (sizeof(T) == 4 ? 4 : 1);
  constexpr int kFetches = LA::kLoads + LB::kLoads;
  constexpr int kEarly = TM > 2 ? TM / 4 : 1;   // rows of products with the fetches among them
  constexpr int kPartTiles = 4;
  __shared__ __align__(1024) char lds[2][(BM + BN) * 128];
  // the epilogue's: room to join the waves, and what it asked for of this item and the next
  __shared__ float2 scratch[Epilogue::kJoins ? WM * BN : 1];
  constexpr int kWanted = Epilogue::template wanted<BM, BN>();
  __shared__ __align__(16) float aside[2][kWanted ? kWanted : 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int items = a.tiles_m * a.tiles_n * a.splits;
  LA la;
  LB lb;
  Place at = place_of(a, blockIdx.x);
  int parity = 0;
  int K;                                        // length of the item's part of k
  const auto begin = [&] {
    const int k0 = at.split * a.part;
    K = min(a.part, a.K - k0);
    la.init(a.a, at.m * BM, k0, lane);
    lb.init(a.b, at.n * BN, k0, lane);
    la.load(lds[0], K, wave);
    lb.load(lds[0] + BM * 128, K, wave);
    la.load(lds[1], K - LA::kBK, wave);
    lb.load(lds[1] + BM * 128, K - LA::kBK, wave);
    at.n0 = a.n0 + at.n * BN;
    ep.template fetch<BM, BN, W>(at, aside[parity], wave, lane);
  };
  begin();
  for (int id = blockIdx.x; id < items;) {
    typename Frag<T>::Sum acc[TM][TN], whole[TM][TN];   // of a part (f32), and of those before it
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = whole[i][j] = typename Frag<T>::Sum{0, 0, 0, 0};
    // Fragments are read half a k-tile ahead of their products, and tiles fetched one and a
    // half ahead, so that the matrix unit has work across the barrier: at it, a wave has
    // read all of the current tile (its buffer may be overwritten) and the next has arrived.
    const int steps = (K + LA::kBK - 1) / LA::kBK;
    typename Frag<T>::V fa[2][TM], fb[2][TN];
    wait_and_meet();
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[0][i] = LA::read(lds[0], (wm * TM + i) * 16, 0, lane);
#pragma unroll
    for (int j = 0; j < TN; ++j)
      fb[0][j] = LB::read(lds[0] + BM * 128, (wn * TN + j) * 16, 0, lane);
    for (int s = 0; s < steps; ++s) {
      char* now = lds[s & 1];
      char* next = lds[(s & 1) ^ 1];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[1][i] = LA::read(now, (wm * TM + i) * 16, 1, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[1][j] = LB::read(now + BM * 128, (wn * TN + j) * 16, 1, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = Frag<T>::mac(fa[0][i], fb[0][j], acc[i][j]);
      interleave<kReads, kMacs>();
      __builtin_amdgcn_sched_barrier(0);
      wait_and_meet();
      const int left = K - (s + 2) * LA::kBK;
#pragma unroll
      for (int i = 0; i < kEarly; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          acc[i][j] = Frag<T>::mac(fa[1][i], fb[1][j], acc[i][j]);
#pragma unroll
          for (int q = (i * TN + j) * kFetches / (kEarly * TN);
               q < (i * TN + j + 1) * kFetches / (kEarly * TN); ++q) {
            if (q < LA::kLoads)
              la.fetch(now, q, left, wave);
            else
              lb.fetch(now + BM * 128, q - LA::kLoads, left, wave);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      la.base += la.step;
      lb.base += lb.step;
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[0][i] = LA::read(next, (wm * TM + i) * 16, 0, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fb[0][j] = LB::read(next + BM * 128, (wn * TN + j) * 16, 0, lane);
#pragma unroll
      for (int i = kEarly; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = Frag<T>::mac(fa[1][i], fb[1][j], acc[i][j]);
      interleave<kReads, kMacs - kEarly * TN * (sizeof(T) == 4 ? 4 : 1)>();
      __builtin_amdgcn_sched_barrier(0);
      if (sizeof(T) == 4 && s % kPartTiles == kPartTiles - 1) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            whole[i][j] += acc[i][j];
            acc[i][j] = typename Frag<T>::Sum{0, 0, 0, 0};
          }
      }
    }
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] += whole[i][j];
    }
    wait_and_meet();   // nothing is on its way, and nobody reads the buffers
    const Place done = at;
    const float* got = aside[parity];
    id += gridDim.x;
    if (id < items) {
      at = place_of(a, id);
      parity ^= 1;
      begin();
    }
    // sums acc[i][j][r]: m = done.m*BM + (wm*TM + i)*16 + (lane>>4)*4 + r,
    //                    n = done.n0 + (wn*TN + j)*16 + (lane&15)
    ep.template run<TM, TN, WM, WN>(acc, done, wm, wn, lane, scratch, got);
  }
}

// Two neighbouring 16 x 16 tiles of a wave's sums as 16-bit values in rows of
// memory: lane (g, c) has rows' places 4g .. 4g+3 of both in column c.  Swapping the
// odd lane groups of the first with the even ones of the second gives every lane
// eight neighbouring values, and a row's 32 values (64 bytes) to the same store:
// half as many requests to the L2 as with eight bytes a lane.
template <typename T>
struct TilePair {
  u32x4 bits;
  static __device__ uint32_t two(float a, float b) {
    typedef T T2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, T2{(T)a, (T)b});
  }
  __device__ TilePair(const f32x4& x, const f32x4& y) {
    const auto a = __builtin_amdgcn_permlane16_swap(two(x[0], x[1]), two(y[0], y[1]), false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(two(x[2], x[3]), two(y[2], y[3]), false, false);
    bits = u32x4{a[0], b[0], a[1], b[1]};
  }
  // where the lane's eight values begin, from the first tile's first row
  static __device__ int at(int g) { return (g & 1) * 16 + (g >> 1) * 8; }
  __device__ void store(T* to) const { *reinterpret_cast<u32x4*>(to) = bits; }
};

// Rows of `width` elements to rows of `padded` (zeros behind them): operands
// whose rows are not 16-byte aligned.  A copy: 5000 rows of 509 bf16 7.4 us, in front of
// 30 of the product at 4000 tokens.
template <typename U>
__global__ __launch_bounds__(256) void pad_kernel(const U* in, int64_t stride, U* out, int64_t rows,
                                                  int32_t width, int32_t padded) {
  const int64_t step = (int64_t)gridDim.x * 256, all = rows * padded;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
    const int64_t r = i / padded;
    const int32_t c = (int32_t)(i % padded);
    out[i] = c < width ? in[r * stride + c] : (U)0;
  }
}

}  // namespace ctcpb_lm
