// A paged key/value cache held in 8 bits, with a scale for each page and head: keys and
// values quantised as they are stored, and read back.
#pragma once
#include <type_traits>

#include "codes.h"

namespace ctcpb_lm {

struct ScaleView {
  float* data;
  int64_t page, head;   // strides in floats
};

struct Cache8Args {
  char *k, *v;                  // read by the store, written by the load
  int64_t k_t, k_h, v_t, v_h;   // strides in bytes
  const int32_t* slots;
  CacheView kc, vc;
  ScaleView ks, vs;
  int32_t tokens, heads, dim;
  int32_t page_log, num_slots;
  int32_t per;                  // pieces of a head's row
  int32_t chunk;                // store: tokens of a wave
};

// Maximum over the wave of `most`, magnitudes of T as Values::raise leaves them.
template <typename T>
__device__ inline uint32_t wave_magnitude(uint32_t most) {
  uint32_t m = Values<T, 1>::magnitude(most);
  for (int x = 1; x < 64; x <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, x));
  return m;
}

// ----------------------------------------------------------------- store --
//
// For the tokens t of the call that go to page p, and head h:
//   scale[p, h] = max(old, least power of two u with max_t |x[t, h]| <= top u)
//   code = nearest code to x / scale
// where old is 0 if a token goes to slot 0 of the page, which begins it anew, else what the
// page has.  Where a page's scale grows, its codes are multiplied by old / new first.
//
// W waves make a page's scale and codes by themselves, so nothing crosses workgroups: tokens of
// one page follow one another in the call, and the waves that have the first of them in their chunk
// of `chunk` tokens (the one before with a slot lies in another page) do the page's whole
// run, for one head of the keys or of the values.  A run's values stay in registers
// between the two passes (maximum, codes) up to kStoreHeld pieces a lane.  W is chosen so that
// those of a page do, up to four waves' 1024 pieces (16 KB of a head); of longer pages, and of those
// that single waves do in calls of few tokens, values that do not fit are read twice.
//
// Bound by memory for prompts: 131072 tokens of 8 x 128 bf16, read and written 805 MB, 163 us in
// pages of 16 (4.9 TB/s; 176 to 186 behind a load), 182 of 32, 176 of 64, 352 of 256, which are
// read twice; a wave to each page of 32 or 64 took 319 and 527.  f32: 292 us in pages of 4, 306 of
// 16, 324 of 64 (1.34 GB, 4.2 to 4.6 TB/s), 556 of 256.  By latency for a step of single tokens, 6
// us for 256.  Where half the registers hold a run, a wave does the keys' and the values' (B = 2
// below): 131072 tokens of 8 x 64 bf16 in pages of 16 91 us; stored and read back 175, against 195
// with a wave to each, and 16 x 32 204 and 268.
constexpr int kStoreHeld = 4;

// The page of the nearest token with a slot before token t, -1 if there is none.
__device__ inline int32_t page_before(const Cache8Args& a, int32_t t, int lane) {
  for (int32_t end = t; end > 0; end -= 64) {
    const int32_t i = end - 64 + lane;
    const int32_t s = i >= 0 ? a.slots[i] : -1;
    const uint64_t in = __ballot((uint32_t)s < (uint32_t)a.num_slots);
    if (in) return __builtin_amdgcn_readlane(s, 63 - __builtin_clzll(in)) >> a.page_log;
  }
  return -1;
}

template <typename T, typename C, int N, int W, int U>
struct StoreRun {
  static constexpr int kLanes = 64 * W, kHeld = U;
  const char* src;          // the head's row of token 0
  int64_t src_t;
  char* page;               // the head's row of slot 0
  int64_t token;
  const int32_t* slots;     // of the run's first token
  int32_t count, num_slots, mask, per;
  int lane;

  // The lane's piece number i: token and piece of its row.
  struct At {
    int32_t t, j;
  };
  __device__ At first() const { return At{lane / per, lane % per}; }
  __device__ void next(At& at) const {
    at.t += kLanes / per;
    at.j += kLanes % per;
    if (at.j >= per) {
      at.j -= per;
      ++at.t;
    }
  }

  Values<T, N> x[U];
  int32_t slot[U];

  // Loads U pieces from `at` on, which moves past them.
  __device__ void load(At& at) {
    At b = at;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      slot[u] = b.t < count ? slots[b.t] : -1;
      next(b);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a token without a slot is not read: it may hold anything
      if ((uint32_t)slot[u] < (uint32_t)num_slots) {
        x[u].load(src + at.t * src_t + at.j * (int)(N * sizeof(T)));
      } else {
        slot[u] = -1;
#pragma unroll
        for (uint32_t& w : x[u].w) w = 0;
      }
      next(at);
    }
  }

  __device__ void raise(uint32_t& most) const {
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].raise(most);
  }

  // Writes the codes of the pieces that load() took from `at` on.
  __device__ void write(At at, float inverse) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (slot[u] >= 0) {
        char* to = page + (slot[u] & mask) * token + at.j * N;
        if constexpr (N == 1) {
          // a scale that is not finite has codes of 0, whatever the values
          const float v = inverse == 0.0f ? 0.0f : x[u].at(0) * inverse;
          *reinterpret_cast<uint8_t*>(to) = (uint8_t)C::round4(v, 0, 0, 0);
        } else {
          uint32_t w[N / 4];
#pragma unroll
          for (int i = 0; i < N / 4; ++i) {
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = x[u].at(4 * i + r) * inverse;
            w[i] = inverse == 0.0f ? 0 : C::round4(v[0], v[1], v[2], v[3]);
          }
          if constexpr (N == 8)
            *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
          else
            *reinterpret_cast<uint32_t*>(to) = w[0];
        }
      }
      next(at);
    }
  }

  // Multiplies the page's codes by `ratio`, a power of two below one.
  __device__ void rescale(float ratio) const {
    At at = first();
    for (; at.t <= mask; next(at)) {
      char* p = page + at.t * token + at.j * N;
      if constexpr (N == 1) {
        float v[4];
        C::values4(*reinterpret_cast<uint8_t*>(p), v);
        *reinterpret_cast<uint8_t*>(p) = (uint8_t)C::round4(v[0] * ratio, 0, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
          uint32_t* q = reinterpret_cast<uint32_t*>(p) + i;
          float v[4];
          C::values4(*q, v);
          *q = C::round4(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
        }
      }
    }
  }
};

// N: values of a piece, 8 (16-bit types) or 4 (f32) where rows and strides allow, else 1.
// W: waves of a workgroup that do a run together; with one, a workgroup's four have four runs.
// B: 2 where half of kStoreHeld is enough: a wave then does the run's keys and values, whose loads
// overlap.
template <typename T, typename C, int N, int W, int B>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void store8_kernel(Cache8Args a) {
  typedef StoreRun<T, C, N, W, kStoreHeld / B> Run;
  __shared__ uint32_t part[2][W];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // (chunk, head, keys or values; with B = 2 both)
  const int64_t unit = (W == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x) * B;
  const int64_t chunk = unit / (2 * a.heads);
  const int64_t begin = chunk * a.chunk;
  if (begin >= a.tokens) return;
  const int32_t head = (int32_t)(unit % (2 * a.heads)) >> 1;
  const int32_t t0 = (int32_t)begin, n = min(a.chunk, a.tokens - t0);

  const int32_t slot = lane < n ? a.slots[t0 + lane] : -1;
  const int32_t prev = t0 > 0 ? a.slots[t0 - 1] : -1;
  const bool in = (uint32_t)slot < (uint32_t)a.num_slots;
  const int32_t mine = in ? slot >> a.page_log : -1;
  const uint64_t all = __ballot(in);
  if (all == 0) return;
  // the page of the token with a slot before the lane's own
  const uint64_t below = all & ((1ull << lane) - 1);
  int32_t before = __shfl(mine, below ? 63 - __builtin_clzll(below) : 0);
  // mostly it is the one right in front of the chunk, asked for along with the chunk's
  const int32_t outside = (uint32_t)prev < (uint32_t)a.num_slots ? prev >> a.page_log
                                                                 : page_before(a, t0 - 1, lane);
  if (!below) before = outside;
  uint64_t leaders = __ballot(in && mine != before);

  const int32_t mask = (1 << a.page_log) - 1;
  for (int parity = 0; leaders; parity ^= 1) {
    const int first = __builtin_ctzll(leaders);
    leaders &= leaders - 1;
    const int32_t page = __builtin_amdgcn_readlane(mine, first);
    // The run: up to the last token of the page before another one begins.
    const uint64_t until = leaders ? (1ull << __builtin_ctzll(leaders)) - 1 : ~0ull;
    const uint64_t same = all & until & ~((1ull << first) - 1);
    int32_t last = t0 + 63 - __builtin_clzll(same), held = __popcll(same);
    bool begun = (__ballot(in && (slot & mask) == 0) & same) != 0;
    if (!leaders) {
      // it may go on past the chunk, for as many tokens as the page has slots
      for (int32_t t = t0 + n; t < a.tokens && held <= mask; t += 64) {
        const int32_t i = t + lane, s = i < a.tokens ? a.slots[i] : -1;
        const uint64_t there = __ballot((uint32_t)s < (uint32_t)a.num_slots);
        const uint64_t other = there & __ballot(s >> a.page_log != page);
        const uint64_t ours = there & (other ? (other & -other) - 1 : ~0ull);
        if (ours) {
          last = t + 63 - __builtin_clzll(ours);
          held += __popcll(ours);
          begun = begun || (ours & __ballot((s & mask) == 0)) != 0;
        }
        if (other) break;
      }
    }
    Run run[B];
    float* scale[B];
    float old[B];
    const int32_t from = t0 + first;
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const bool values = B == 2 ? b : unit & 1;
      const CacheView& c = values ? a.vc : a.kc;
      const ScaleView& sc = values ? a.vs : a.ks;
      Run& r = run[b];
      r.src_t = values ? a.v_t : a.k_t;
      r.src = (values ? a.v + head * a.v_h : a.k + head * a.k_h) + from * r.src_t;
      r.page = c.data + page * c.page + head * c.head;
      r.token = c.token;
      r.slots = a.slots + from;
      r.count = last - from + 1;
      r.num_slots = a.num_slots;
      r.mask = mask;
      r.per = a.per;
      r.lane = W == 1 ? lane : (int)threadIdx.x;
      scale[b] = sc.data + page * sc.page + head * sc.head;
      old[b] = begun ? 0.0f : *scale[b];
    }
    const int64_t pieces = (int64_t)run[0].count * a.per;
    const int64_t batches = (pieces + Run::kLanes * Run::kHeld - 1) / (Run::kLanes * Run::kHeld);
    typename Run::At at = run[0].first();
    const auto at0 = at;
    uint32_t most[B] = {};
    for (int64_t i = 0; i < batches; ++i) {
      const auto here = at;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        at = here;
        run[b].load(at);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) run[b].raise(most[b]);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) most[b] = wave_magnitude<T>(most[b]);
    if constexpr (W > 1) {
      static_assert(B == 1, "a wave's own");
      if (lane == 0) part[parity][wave] = most[0];
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) most[0] = max(most[0], part[parity][w]);
    }
    float now[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const float need = bits_f32(unit_bits<C>(most[b])), was = old[b];
      // (a NaN stays, whichever of the two it is)
      now[b] = was != was ? was : need != need || need > was ? need : was;
      if (now[b] > was && was > 0.0f) {
        run[b].rescale(was / now[b]);
        // the new codes go over some of these
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if constexpr (W > 1) __syncthreads();
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const float inverse = inverse_unit(now[b]);
      if (batches == 1) {
        run[b].write(at0, inverse);
      } else {
        at = at0;
        for (int64_t i = 0; i < batches; ++i) {
          const auto here = at;
          run[b].load(at);
          run[b].write(here, inverse);
        }
      }
      if (run[b].lane == 0) *scale[b] = now[b];
    }
  }
}

// ------------------------------------------------------------------ load --
//
// k[t, h] = code * scale of the token's slot, in T; zeros for a token without a slot.  A copy,
// bound by memory: 131072 tokens of 8 x 128 to bf16 162 us, 5.0 TB/s, to f32 320 (4.2); 500 of 8 x
// 64 to f32 3.4 us.  A thread makes 16 bytes of a key's row, then the same of the value's: with both
// rows' codes asked for before either is stored, times hang on where the tensors lie (155 or 171 us
// to bf16, 267 or 342 to f32).  A thread's first piece is found by divisions in 32 bits: in 64 they
// took 7 us more.
//
// What is finite is read as such: the nearest code to a value next to the type's largest one may
// stand for more (f16 65504 in int8 is 64 * 1024), and is read as the largest.  No code reaches
// 512, so only scales above a 512th of that have to be looked at, in a branch of the whole wave.
template <typename T, typename C, int N>
__global__ __launch_bounds__(256) void load8_kernel(Cache8Args a) {
  const uint32_t row = (uint32_t)(a.heads * a.per), step = gridDim.x * 256;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;   // (2^28 threads at most)
  uint32_t t = i / row, rest = i % row;
  for (; t < (uint32_t)a.tokens; t += step / row, rest += step % row) {
    if (rest >= row) {
      rest -= row;
      if (++t >= (uint32_t)a.tokens) break;
    }
    const int32_t h = (int32_t)(rest / (uint32_t)a.per), p = (int32_t)(rest % (uint32_t)a.per);
    const int32_t slot = a.slots[t];
    const bool in = (uint32_t)slot < (uint32_t)a.num_slots;
    const int64_t page = in ? slot >> a.page_log : 0, at = slot & ((1 << a.page_log) - 1);
    constexpr int W = N == 1 ? 1 : N / 4;
    constexpr float most = kLargest<T>;
    // (0 times a scale of 0 without a slot)
    float scale[2] = {0.0f, 0.0f};
    if (in) {
      scale[0] = a.ks.data[page * a.ks.page + h * a.ks.head];
      scale[1] = a.vs.data[page * a.vs.page + h * a.vs.head];
    }
    const auto load = [&](int half, uint32_t (&w)[W]) {
#pragma unroll
      for (uint32_t& x : w) x = 0;
      if (!in) return;
      const CacheView& c = half ? a.vc : a.kc;
      const char* from = c.data + page * c.page + at * c.token + h * c.head + p * N;
      if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint8_t*>(from);
      } else if constexpr (N == 8) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(from);
        w[0] = x[0];
        w[1] = x[1];
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(from);
      }
    };
    const auto store = [&](int half, const uint32_t (&w)[W], auto limit) {
      T out[N];
#pragma unroll
      for (int b = 0; b < W; ++b) {
        float v[4];
        C::values4(w[b], v);
#pragma unroll
        for (int r = 0; r < 4 && r < N; ++r) {
          float x = v[r] * scale[half];
          if (limit && fabsf(scale[half]) < bits_f32(kInfBits))
            x = x > most ? most : x < -most ? -most : x;   // (a NaN stays)
          out[4 * b + r] = (T)x;
        }
      }
      T* to = reinterpret_cast<T*>((half ? a.v + t * a.v_t + h * a.v_h
                                         : a.k + t * a.k_t + h * a.k_h)) + p * N;
      if constexpr (N == 1) {
        *to = out[0];
      } else {
        static_assert(N * sizeof(T) == 16, "a piece is 16 bytes");
        *reinterpret_cast<u32x4*>(to) = __builtin_bit_cast(u32x4, out);
      }
    };
    uint32_t w[W];
    load(0, w);
    if (__any(fmaxf(fabsf(scale[0]), fabsf(scale[1])) > most / 512.0f)) {
      store(0, w, std::true_type{});
      load(1, w);
      store(1, w, std::true_type{});
    } else {
      store(0, w, std::false_type{});
      load(1, w);
      store(1, w, std::false_type{});
    }
  }
}

}  // namespace ctcpb_lm
