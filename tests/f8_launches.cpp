// Host replay of the launches of dropout and of the linear layer in 8-bit
// floating point (built host-only by test_f8_launches.py; no GPU is needed and
// no kernel runs).
//
// The program stands in for the few runtime functions that the library calls:
// it reports a gfx950 device, notes every kernel that the library registers
// and, instead of launching one, replays from its arguments the addresses that
// its threads form.  Operands and workspaces are ranges of made-up addresses
// with their exact extents, so an access outside of all of them is found, and
// so is an offset that does not fit the 32 bits the kernels keep it in.  The
// expressions mirror quant_f8.hip, gemm_f8.h, linear_f8.hip and dropout.hip.
#include <cxxabi.h>
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <map>
#include <set>
#include <string>
#include <vector>

#include "../post_pruning_amd/csrc/gemm_f8.h"

using sg::F8Args;
using sg::NtArgs;

namespace {

struct Range {
  const char* name;
  uint64_t at, bytes;
};
std::vector<Range> ranges;  // the call's output is the first
int failures = 0;
std::string what, kernel;

void fail(const char* fmt, ...) {
  if (++failures > 10) return;
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  fprintf(stderr, "FAIL %s: %s: %s\n", what.c_str(), kernel.substr(0, 80).c_str(), buf);
}

uint8_t* make(const char* name, uint64_t bytes, uint64_t shift = 0) {
  const uint64_t at = ((uint64_t)ranges.size() + 1) << 56;
  ranges.push_back({name, at + shift, bytes});
  return reinterpret_cast<uint8_t*>(at + shift);
}

template <typename P>
void touch(const char* who, P* p, int64_t off, uint64_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p) + (uint64_t)off;
  for (const Range& r : ranges)
    if (at >= r.at && at + bytes <= r.at + r.bytes) return;
  const uint64_t k = at >> 56;
  if (k >= 1 && k <= ranges.size())
    fail("%s: byte %lld of '%s', which has %lld", who, (long long)(at - ranges[k - 1].at), ranges[k - 1].name,
         (long long)ranges[k - 1].bytes);
  else
    fail("%s: address %llx is in no operand", who, (unsigned long long)at);
}

// An offset that a kernel keeps in 32 bits.
int64_t in32(const char* who, int64_t off) {
  if (off < 0 || off >= (int64_t)1 << 32) fail("%s: offset %lld does not fit 32 bits", who, (long long)off);
  return off;
}
void inside(const char* who, int64_t at, int64_t bytes, int64_t size) {
  if (at < 0 || at + bytes > size) fail("%s: LDS bytes %lld + %lld of %lld", who, (long long)at, (long long)bytes, (long long)size);
}
void shape(bool ok, dim3 grid, dim3 block) {
  if (!ok) fail("grid %u x %u, block %u x %u", grid.x, grid.y, block.x, block.y);
  if ((uint64_t)grid.x * grid.y * block.x * block.y >= (uint64_t)1 << 32) fail("2^32 threads or more");
  if (grid.y > 65535) fail("grid of %u rows", grid.y);
}

// The first, the last and one between them.
std::vector<int64_t> some(int64_t n) {
  std::set<int64_t> s;
  for (int64_t i : {(int64_t)0, n / 2, n - 1})
    if (i >= 0 && i < n) s.insert(i);
  return {s.begin(), s.end()};
}
std::vector<int> stages(int n, int ring) {
  std::set<int> s;
  for (int i : {0, ring, n - 2, n - 1})
    if (i >= 0 && i < n) s.insert(i);
  return {s.begin(), s.end()};
}

std::map<std::string, int> seen;
int64_t rows_done;  // of the call's first dimension, in launches that follow each other

void next_rows(const void* at, int64_t pitch, int64_t rows) {
  if (rows < 1 || reinterpret_cast<uint64_t>(at) != ranges[0].at + rows_done * pitch) fail("rows left out after %lld", (long long)rows_done);
  rows_done += rows;
}

// How far into its operand a pointer points.
template <typename P>
int64_t into(P* p) {
  const uint64_t at = reinterpret_cast<uint64_t>(p), k = at >> 56;
  return k >= 1 && k <= ranges.size() ? (int64_t)(at - ranges[k - 1].at) : -1;
}

template <typename T>
const T& arg(void** a, int i) {
  return *static_cast<const T*>(a[i]);
}

// What a kernel's name says between its first '<' and the parameters.
std::vector<std::string> words() {
  std::vector<std::string> v;
  std::string w;
  const size_t from = kernel.find("_kernel<");
  for (size_t i = from == std::string::npos ? kernel.size() : from + 8; i < kernel.size() && kernel[i] != '('; ++i) {
    const char c = kernel[i];
    if (c == ',' || c == '<' || c == '>') {
      if (!w.empty()) v.push_back(w);
      w.clear();
    } else if (c != ' ') {
      w += c;
    }
  }
  return v;
}
int number(const std::vector<std::string>& v, size_t i) {
  return i >= v.size() ? 0 : v[i] == "true" ? 1 : v[i] == "false" ? 0 : atoi(v[i].c_str());
}
int64_t element(const std::vector<std::string>& v) { return !v.empty() && v[0] == "float" ? 4 : 2; }

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
struct Tile {
  int wide, TA, TB, WA, WB, R, split;
  int waves() const { return WA * WB; }
  int threads() const { return 64 * waves(); }
  int FA() const { return TA / WA / 16; }
  int FB() const { return TB / WB / 16; }
};
Tile tile_of() {
  const std::vector<std::string> v = words();  // sg::F8Tile, WIDE, E5, TA, TB, WA, WB, R, SPLIT
  return Tile{number(v, 1), number(v, 3), number(v, 4), number(v, 5), number(v, 6), number(v, 7), number(v, 8)};
}

// F8Tile's copies of the stages [s0, s0 + n)
void tile_copies(const Tile& t, const F8Args& p, int64_t a0, int64_t b0, int s0, int n) {
  const NtArgs& g = p.g;
  const int CA = t.TA / 8 / t.waves(), CB = t.TB / 8 / t.waves();
  const int64_t astage = t.TA * 128, stage = astage + t.TB * 128;
  for (int tid = 0; tid < t.threads(); ++tid) {
    const int wave = tid / 64, lane = tid % 64, r = wave * 8 + (lane >> 3);
    const int chunk = std::min(wave, (t.TA + t.TB) / 64 - 1);
    const bool of_b = chunk >= t.TA / 64;
    const int64_t first = of_b ? b0 + 64 * (chunk - t.TA / 64) : a0 + 64 * chunk;
    const int64_t pitch = of_b ? p.b_lds : p.a_lds;
    const int64_t off_s = in32("scales", std::min<int64_t>(first + (lane & 15) * 4, ((of_b ? g.nb : g.na) - 1) & ~(int64_t)3));
    inside("scales", wave * 256 + lane * 4, 4, t.waves() * 256);
    const int64_t last_a = in32("A", (std::min<int64_t>(t.TA, g.na - a0) - 1) * g.lda);
    const int64_t last_b = in32("B", (std::min<int64_t>(t.TB, g.nb - b0) - 1) * g.ldb);
    for (int s : stages(n, t.R)) {
      touch("scales", (of_b ? p.b_scale : p.a_scale) + (s0 + s) * pitch, off_s, 4);
      for (int k = 0; k < CA; ++k) {
        const int rk = r + 8 * t.waves() * k, piece = (lane & 7) ^ (2 * ((rk >> 4) & 3) + ((rk >> 1) & 1));
        const int64_t off = std::min(in32("A", r * g.lda) + in32("A", k * 8 * t.waves() * g.lda), last_a) + piece * 16;
        touch("A", g.A + a0 * g.lda + (int64_t)(s0 + s) * 128, in32("A", off), 16);
        inside("A", (t.waves() * k + wave) * 1024 + lane * 16, 16, astage);
      }
      for (int k = 0; k < CB; ++k) {
        const int64_t off = std::min(in32("B", r * g.ldb) + in32("B", k * 8 * t.waves() * g.ldb), last_b) +
                            ((lane & 7) ^ ((r >> 1) & 7)) * 16;
        touch("B", g.B + b0 * g.ldb + (int64_t)(s0 + s) * 128, in32("B", off), 16);
        inside("B", astage + (t.waves() * k + wave) * 1024 + lane * 16, 16, stage);
      }
    }
  }
}

void store(const NtArgs& g, int64_t a, int64_t b, int width) {
  if (b >= g.nb || a >= g.na) return;
  const int64_t e = g.out_dtype == SG_F32 ? 4 : 2, cnt = std::min<int64_t>(g.na - a, width);
  touch("out", static_cast<char*>(g.out), (b * g.ldo + a) * e, cnt * e);
  if (g.mask) touch("mask", g.mask, b * g.na + a, cnt);
}
void tile_outputs(const Tile& t, const NtArgs& g, int64_t a0, int64_t b0, int q) {  // item q of every wave
  for (int tid = 0; tid < t.threads(); ++tid) {
    const int wave = tid / 64, lane = tid % 64;
    store(g, a0 + (wave / t.WB) * (t.TA / t.WA) + (q / t.FB()) * 64 + (lane >> 4) * 16,
          b0 + (wave % t.WB) * (t.TB / t.WB) + (q % t.FB()) * 16 + (lane & 15), 16);
  }
}

void replay_tiles(void** a, dim3 grid, dim3 block) {
  const Tile t = tile_of();
  const F8Args& p = arg<F8Args>(a, 0);
  const NtArgs& g = p.g;
  const int64_t ta = arg<int64_t>(a, 1), tb = arg<int64_t>(a, 2);
  const int splits = arg<int>(a, 3);
  sg::floatx4* const part = arg<sg::floatx4*>(a, 4);
  shape((int)block.x == t.threads() && (int64_t)grid.x >= ta * tb * splits && grid.x % 8 == 0, grid, block);
  if (ta != sg::ceil_div(g.na, t.TA) || tb != sg::ceil_div(g.nb, t.TB)) fail("%lld x %lld tiles", (long long)ta, (long long)tb);
  if (t.wide != (g.out_dtype == SG_F32)) fail("the output's type and the tile's");
  if (!t.split && splits != 1) fail("%d splits of whole tiles", splits);
  // a launch of later rows takes them of every operand
  if (p.row0 != rows_done || into(g.B) != rows_done * g.ldb || into(p.b_scale) != rows_done || into(g.A) != 0 ||
      into(p.a_scale) != 0 || (g.mask && into(g.mask) != rows_done * g.na))
    fail("operands of the rows from %lld on", (long long)rows_done);
  next_rows(g.out, g.ldo * (g.out_dtype == SG_F32 ? 4 : 2), g.nb);
  const int steps = (int)(g.kbytes / 128);
  for (int64_t ia : some(ta))
    for (int64_t ib : some(tb))
      for (int64_t sp : some(splits)) {
        const int s0 = (int)((int64_t)steps * sp / splits), s1 = (int)((int64_t)steps * (sp + 1) / splits);
        if (s1 > s0) tile_copies(t, p, ia * t.TA, ib * t.TB, s0, s1 - s0);
        const int64_t slots = (int64_t)t.FA() * t.FB() * t.threads();
        if (t.split)  // the tile's number takes every value below ta tb
          for (int64_t k : {(int64_t)0, ta * tb - 1}) touch("partial sums", part, (k * splits + sp) * slots * 16, slots * 16);
        else
          for (int q = 0; q < t.FA() / 4 * t.FB(); ++q) tile_outputs(t, g, ia * t.TA, ib * t.TB, q);
      }
}

void replay_join(void** a, dim3 grid, dim3 block) {
  const Tile t = tile_of();
  const NtArgs& g = arg<F8Args>(a, 0).g;
  const int64_t ta = arg<int64_t>(a, 1), tb = arg<int64_t>(a, 2);
  const int64_t slots = (int64_t)t.FA() * t.FB() * t.threads();
  shape((int64_t)grid.x == ta * tb && (int)grid.y == t.FA() / 4 * t.FB() && (int)block.x == t.threads(), grid, block);
  touch("partial sums", arg<sg::floatx4*>(a, 4), 0, ta * tb * arg<int>(a, 3) * slots * 16);
  for (int64_t ia : some(ta))
    for (int64_t ib : some(tb))
      for (int q = 0; q < (int)grid.y; ++q) tile_outputs(t, g, ia * t.TA, ib * t.TB, q);
}

void replay_stream(void** a, dim3 grid, dim3 block) {
  const F8Args& p = arg<F8Args>(a, 0);
  const NtArgs& g = p.g;
  const std::vector<std::string> v = words();  // WIDE, E5, CF, TF, W, U
  const int CF = number(v, 2), TF = number(v, 3), W = number(v, 4), steps = (int)(g.kbytes / 128);
  shape((int)block.x == 64 * W && (int64_t)grid.x * 16 * CF >= g.na && g.nb <= 16 * TF, grid, block);
  if (CF * TF * W * 1024 > 160 * 1024) fail("sums in LDS");
  next_rows(g.out, g.ldo * (g.out_dtype == SG_F32 ? 4 : 2), g.nb);
  for (int64_t wg : some(grid.x))
    for (int lane = 0; lane < 64; ++lane) {
      const int64_t a0 = wg * 16 * CF;
      for (int c = 0; c < CF; ++c) {
        const int64_t r = std::min<int64_t>(a0 + 16 * c + (lane & 15), g.na - 1);
        for (int s : stages(steps, 2)) {
          for (int h : {0, 64}) touch("A", g.A, r * g.lda + (lane >> 4) * 16 + (int64_t)s * 128 + h, 16);
          touch("A's scales", p.a_scale, s * p.a_lds + r, 1);
        }
      }
      for (int f = 0; f < TF; ++f) {
        const int64_t r = std::min<int64_t>(16 * f + (lane & 15), g.nb - 1);
        for (int s : stages(steps, 2)) {
          for (int h : {0, 64}) touch("B", g.B, r * g.ldb + (lane >> 4) * 16 + (int64_t)s * 128 + h, 16);
          touch("B's scales", p.b_scale, s * p.b_lds + r, 1);
        }
        for (int c = 0; c < CF; ++c) store(g, a0 + 16 * c + (lane >> 4) * 4, 16 * f + (lane & 15), 4);
      }
    }
}

// ---------------------------------------------------------------------------
// Quantizers and dropout
// ---------------------------------------------------------------------------
struct Out {  // as in quant_f8.hip
  uint8_t* q;
  int64_t ldq;
  uint8_t* scale;
  int64_t lds;
};

// load8 of columns [c0, c0 + 8) of a row at `row`
void load8(const uint8_t* row, int64_t c0, int64_t n, int64_t e) {
  if (c0 + 8 <= n)
    touch("X", row, c0 * e, 8 * e);
  else
    for (int k = 0; k < 8; ++k) touch("X", row, std::min(c0 + k, n - 1) * e, e);
}

void replay_rows(void** a, dim3 grid, dim3 block) {
  const std::vector<std::string> v = words();
  const int64_t e = element(v);
  uint8_t *q = arg<uint8_t*>(a, 0), *scale = arg<uint8_t*>(a, 2);
  const int64_t ldq = arg<int64_t>(a, 1), lds = arg<int64_t>(a, 3), T = arg<int64_t>(a, 5), n = arg<int64_t>(a, 6),
                ldx = arg<int64_t>(a, 7);
  const uint8_t* X = arg<uint8_t*>(a, 4);
  shape(block.x == 256 && (int64_t)grid.x == sg::ceil_div(n, 128) && grid.y >= 1, grid, block);
  next_rows(q, ldq, T);
  for (int64_t kb : some(grid.x))
    for (int tid = 0; tid < 256; ++tid)
      for (int64_t t : some(T)) {
        if (t % 16 != tid >> 4) continue;
        const int64_t c0 = kb * 128 + (tid & 15) * 8;
        load8(X + t * ldx * e, c0, n, e);
        touch("Q", q, t * ldq + c0, 8);
        touch("scale", scale, kb * lds + t, 1);
      }
}

void replay_tile_quantizer(void** a, dim3 grid, dim3 block) {
  const std::vector<std::string> v = words();
  const int64_t e = element(v);
  const bool drop = number(v, 2);
  const Out &rows = arg<Out>(a, 0), &cols = arg<Out>(a, 1);
  const uint8_t* X = arg<uint8_t*>(a, 2);
  const int64_t T = arg<int64_t>(a, 3), n = arg<int64_t>(a, 4), ldx = arg<int64_t>(a, 5), kn = arg<int64_t>(a, 6), row0 = arg<int64_t>(a, 8);
  shape(block.x == 512 && kn == sg::ceil_div(n, 128) && (int64_t)grid.x == sg::ceil_div(T, 128) * kn, grid, block);
  if (drop && row0 != rows_done) fail("the first row's number");
  if ((rows.q && (into(rows.q) != rows_done * rows.ldq || into(rows.scale) != rows_done)) ||
      (cols.q && (into(cols.q) != rows_done || into(cols.scale) != rows_done / 128 * cols.lds)))
    fail("outputs of the rows from %lld on", (long long)rows_done);
  if (reinterpret_cast<uint64_t>(X) != ranges[0].at + rows_done * ldx * e) fail("rows left out after %lld", (long long)rows_done);
  rows_done += T;
  for (int64_t kt : some(sg::ceil_div(T, 128)))
    for (int64_t kc : some(kn))
      for (int tid = 0; tid < 512; ++tid) {
        const int64_t c0 = kc * 128 + (tid & 15) * 8, t0 = kt * 128 + (tid >> 4) * 4;
        for (int k = 0; k < 4; ++k) {
          if (t0 + k >= T) continue;
          load8(X + (t0 + k) * ldx * e, c0, n, e);
          if (rows.q) {
            touch("rows", rows.q, (t0 + k) * rows.ldq + c0, 8);
            touch("scales of rows", rows.scale, kc * rows.lds + t0 + k, 1);
          }
        }
        if (!cols.q) continue;
        if (tid < 16)
          for (int64_t c = c0; c < std::min(c0 + 8, n); ++c) touch("scales of columns", cols.scale, kt * cols.lds + c, 1);
        for (int i = 0; i < 4; ++i) {
          const int64_t c = 32 * i + (tid >> 4);
          if (kc * 128 + c < n) touch("columns", cols.q, (kc * 128 + c) * cols.ldq + kt * 128 + (tid & 15) * 8, 8);
        }
      }
}

void replay_values(void** a, dim3 grid, dim3 block) {
  const int64_t e = element(words());
  uint8_t *X = arg<uint8_t*>(a, 0), *q = arg<uint8_t*>(a, 2), *scale = arg<uint8_t*>(a, 4);
  const int64_t ldx = arg<int64_t>(a, 1), ldq = arg<int64_t>(a, 3), lds = arg<int64_t>(a, 5), T = arg<int64_t>(a, 6), n = arg<int64_t>(a, 7);
  shape(block.x * block.y == 256 && (int64_t)grid.x * block.x * 16 >= n, grid, block);
  next_rows(X, ldx * e, T);
  for (int64_t t : some(T))
    for (int64_t c : some(sg::ceil_div(n, 16))) {
      touch("Q", q, t * ldq + 16 * c, 16);
      touch("scale", scale, 16 * c / 128 * lds + t, 1);
      touch("X", X, (t * ldx + 16 * c) * e, std::min<int64_t>(16, n - 16 * c) * e);
    }
}

void replay_dropout(void** a, dim3 grid, dim3 block) {
  const std::vector<std::string> v = words();
  const int64_t e = element(v);
  const int64_t ldy = arg<int64_t>(a, 1), ldx = arg<int64_t>(a, 3), ldr = arg<int64_t>(a, 5), T = arg<int64_t>(a, 6), n = arg<int64_t>(a, 7);
  shape(block.x * block.y == 256 && (int64_t)grid.x * block.x * 8 >= n, grid, block);
  next_rows(arg<uint8_t*>(a, 0), ldy * e, T);
  for (int64_t t : some(T))
    for (int64_t c : some(sg::ceil_div(n, 8))) {
      const int64_t bytes = std::min<int64_t>(8, n - 8 * c) * e;
      touch("Y", arg<uint8_t*>(a, 0), (t * ldy + 8 * c) * e, bytes);
      touch("X", arg<uint8_t*>(a, 2), (t * ldx + 8 * c) * e, bytes);
      if (number(v, 1)) touch("residual", arg<uint8_t*>(a, 4), (t * ldr + 8 * c) * e, bytes);
    }
}

void replay(void** a, dim3 grid, dim3 block) {
  auto is = [](const char* n) { return kernel.find(std::string("sg::") + n + "<") != std::string::npos; };
  if (is("f8_tiles_kernel"))
    replay_tiles(a, grid, block);
  else if (is("f8_join_kernel"))
    replay_join(a, grid, block);
  else if (is("f8_stream_kernel"))
    replay_stream(a, grid, block);
  else if (is("f8_rows_kernel"))
    replay_rows(a, grid, block);
  else if (is("f8_tile_kernel"))
    replay_tile_quantizer(a, grid, block);
  else if (is("f8_values_kernel"))
    replay_values(a, grid, block);
  else if (is("dropout_kernel"))
    replay_dropout(a, grid, block);
  else
    fail("unknown kernel");
}

std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
struct Config {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
} config;

}  // namespace

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*, int*) {
  int status = 0;
  char* d = abi::__cxa_demangle(device, nullptr, nullptr, &status);
  std::string name = d ? d : device;
  free(d);
  const std::string anon = "(anonymous namespace)::";
  for (size_t at; (at = name.find(anon)) != std::string::npos;) name.erase(at, anon.size());
  names()[host] = name;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  config = Config{grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = config.grid, *block = config.block, *shared = config.shared, *stream = config.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  kernel = names().count(f) ? names()[f] : "?";
  ++seen[kernel.substr(0, kernel.find('('))];
  replay(args, grid, block);
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  memset(p, 0, sizeof(*p));
  strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
}

// ---------------------------------------------------------------------------
// Calls
// ---------------------------------------------------------------------------
namespace {

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Codes and scale bytes of a matrix, with rows `far` bytes further apart than they need.
Out codes(const char* name, int64_t rows, int64_t cols, int64_t far = 0) {
  Out o;
  o.ldq = std::min<int64_t>(up(cols, 128) + far, (int64_t)1 << 23);
  o.lds = up(rows, 16);
  o.q = make(name, rows > 0 ? (rows - 1) * o.ldq + up(cols, 128) : 0);
  o.scale = make("scale bytes", up(cols, 128) / 128 * o.lds);
  return o;
}
uint8_t* matrix(const char* name, int64_t rows, int64_t cols, int64_t ld, int64_t e, int64_t shift) {
  return make(name, rows > 0 ? ((rows - 1) * ld + cols) * e : 0, shift * e);
}

void begin(const char* call, int64_t T, int64_t n, int64_t m) {
  ranges.clear();
  rows_done = 0;
  kernel = "-";
  char buf[200];
  snprintf(buf, sizeof(buf), "%s T=%lld n=%lld m=%lld", call, (long long)T, (long long)n, (long long)m);
  what = buf;
}
void expect_ok(sg_status s, int64_t rows) {
  if (s != SG_OK) fail("status %d: %s", (int)s, sg_last_error_message());
  if (rows_done != rows) fail("%lld of %lld rows", (long long)rows_done, (long long)rows);
}

const sg_drop kDrop = {0.25, 1, 2, nullptr};

void products(int64_t T, int64_t n, int64_t m, int dtype, int64_t far = 0, int64_t extra = 0, int64_t shift = 0) {
  const int64_t e = dtype == SG_F32 ? 4 : 2;
  auto space = [&](int32_t op) { return sg_workspace_bytes(op, m, n, T, 0); };
  {
    begin("linear", T, n, m);
    uint8_t* Y = matrix("Y", T, m, m + extra, e, shift);
    const Out q = codes("Q", T, n, far), w = codes("W", m, n, far);
    const size_t nb = space(SG_OP_LINEAR_F8);
    expect_ok(sg_linear_f8(Y, dtype, m + extra, q.q, q.ldq, q.scale, q.lds, T % 2, T, w.q, w.ldq, w.scale, w.lds, m, n,
                           make("workspace", nb), nb, nullptr), T);
  }
  {
    begin("grad_input", T, n, m);
    uint8_t* dX = matrix("dX", T, n, n + extra, e, shift);
    const Out q = codes("dY", T, m, far), w = codes("Wt", n, m, far);
    const size_t nb = space(SG_OP_F8_GRAD_INPUT);
    expect_ok(sg_linear_f8_grad_input(dX, dtype, n + extra, q.q, q.ldq, q.scale, q.lds, T % 2, T, w.q, w.ldq, w.scale,
                                      w.lds, m, n, T % 3 ? &kDrop : nullptr, make("workspace", nb), nb, nullptr), T);
  }
  if (T > 1 << 23) return;
  {
    begin("grad_weight", T, n, m);
    uint8_t* dW = matrix("dW", m, n, n + extra, e, shift);
    const Out q = codes("dYt", m, T, far), x = codes("Xt", n, T, far);
    const size_t nb = space(SG_OP_F8_GRAD_WEIGHT);
    uint8_t* mask = T % 2 ? make("mask", m * n, shift) : nullptr;
    expect_ok(sg_linear_f8_grad_weight(dW, dtype, n + extra, 0, q.q, q.ldq, q.scale, q.lds, T % 2, x.q, x.ldq, x.scale,
                                       x.lds, T, mask, m, n, make("workspace", nb), nb, nullptr), m);
  }
}

void quantizers(int64_t T, int64_t n, int dtype, int64_t extra = 0, int64_t shift = 0) {
  const int64_t e = dtype == SG_F32 ? 4 : 2;
  {
    begin("quantize rows", T, n, 0);
    const Out q = codes("Q", T, n);
    uint8_t* X = matrix("X", T, n, n + extra, e, shift);
    expect_ok(sg_quantize_f8(q.q, q.ldq, q.scale, q.lds, nullptr, 0, nullptr, 0, T % 2, X, dtype, T, n, n + extra,
                             T % 3 ? &kDrop : nullptr, nullptr), T);
  }
  {
    begin("read back", T, n, 0);
    uint8_t* X = matrix("X", T, n, n + extra, e, shift);
    const Out q = codes("Q", T, n);
    expect_ok(sg_dequantize_f8(X, dtype, n + extra, q.q, q.ldq, q.scale, q.lds, T % 2, T, n, nullptr), T);
  }
  {
    begin("dropout", T, n, 0);
    uint8_t* Y = matrix("Y", T, n, n + extra, e, shift);
    uint8_t* X = matrix("X", T, n, n + extra, e, shift);
    uint8_t* R = T % 2 ? matrix("R", T, n, n, e, 0) : nullptr;
    expect_ok(sg_dropout(Y, n + extra, X, dtype, n + extra, R, n, T, n, &kDrop, nullptr), T);
  }
  for (int both = 0; both < 2 && T <= 1 << 23; ++both) {
    begin("quantize columns", T, n, 0);
    uint8_t* X = matrix("X", T, n, n + extra, e, shift);
    const Out none{}, q = both ? codes("Q", T, n) : none, c = codes("Qt", n, T);
    expect_ok(sg_quantize_f8(q.q, q.ldq, q.scale, q.lds, c.q, c.ldq, c.scale, c.lds, T % 2, X, dtype, T, n, n + extra,
                             T % 3 ? &kDrop : nullptr, nullptr), T);
  }
  if (n > 65536 || T > 1 << 20) return;
  for (int both = 0; both < 2; ++both) {
    begin("pack", T, n, 0);
    uint8_t* W = matrix("W", T, n, n + extra, e, shift);
    const Out w = codes("W", T, n), none{}, t = both ? codes("Wt", n, T) : none;
    expect_ok(sg_pack_f8(w.q, w.ldq, w.scale, w.lds, t.q, t.ldq, t.scale, t.lds, W, dtype, T, n, n + extra, nullptr), T);
  }
}

struct Sizes {
  int64_t T, n, m;
};
const Sizes kShapes[] = {
    {1, 1, 1},         {1, 4096, 4096},   {2, 130, 70},       {16, 1000, 520},    {16, 28672, 8192},   {17, 257, 100},
    {31, 11008, 700},  {33, 4100, 130},   {48, 2048, 2048},   {64, 512, 300},     {65, 640, 257},      {100, 128, 1000},
    {130, 129, 385},   {200, 8200, 203},  {257, 1100, 511},   {300, 1000, 1130},  {512, 4096, 768},    {515, 300, 2050},
    {512, 4096, 4096}, {1030, 520, 1300}, {2048, 1024, 2048}, {2500, 384, 4099},  {4100, 200, 140},    {8192, 4096, 11008},
    {1, 4096, 11008},  {513, 4096, 768},  {1023, 2000, 4100}, {2049, 1024, 2048}, {4711, 4424, 68},   {4712, 4424, 68},
    {69, 5735, 4490},  {70, 5735, 4490},  {69, 7457, 8223},   {70, 7457, 8223},   {77, 35851, 4489},  {78, 35851, 4489},
    {4587, 58543, 139}, {4588, 58543, 139}, {10, 28672, 8192}, {10, 4096, 11008}, {10, 1000, 520},    {9, 28672, 8192},
    {65, 2509, 3},     {66, 4300, 5},     {8191, 4095, 1},   {20001, 203, 8200}, {70000, 64, 64},   {300, 65536, 1 << 20}};

void shapes() {
  for (const Sizes& s : kShapes)
    for (int dtype : {SG_F32, SG_BF16}) {
      products(s.T, s.n, s.m, dtype);
      products(s.T, s.n, s.m, dtype, 128, 3, 1);
      quantizers(s.T, s.n, dtype);
      quantizers(s.T, s.n, dtype, 5, 1);
    }
}
// rows as far apart as they may lie
void pitches() {
  for (const Sizes& s : {Sizes{5, 300, 520}, Sizes{300, 1000, 700}, Sizes{2500, 384, 4099}, Sizes{1030, 8000, 4100}})
    for (int dtype : {SG_F32, SG_BF16}) products(s.T, s.n, s.m, dtype, (int64_t)1 << 23);
}
// up to the largest sizes
void many() {
  const int64_t top = ((int64_t)1 << 31) - 1;
  for (int dtype : {SG_F32, SG_BF16}) {
    products((int64_t)1 << 23, 300, 700, dtype);
    products(((int64_t)1 << 23) - 5, 65536, 130, dtype);
    products(top, 200, 1000, dtype);
    products(top - 1, 65536, 1 << 16, dtype);
    quantizers((int64_t)1 << 23, 1, dtype);
    quantizers(((int64_t)1 << 23) - 200, 1 << 20, dtype);
    quantizers(top, 1, dtype);
    quantizers(top - 1, 1 << 20, dtype);
    quantizers(300, 1 << 20, dtype);
    quantizers(1 << 20, 65536, dtype);
  }
}

}  // namespace

int main(int argc, char** argv) {
  const std::string test = argc > 1 ? argv[1] : "";
  if (test == "shapes")
    shapes();
  else if (test == "pitches")
    pitches();
  else if (test == "many")
    many();
  else
    return 2;
  for (const auto& k : seen) printf("%6d %s\n", k.second, k.first.c_str());
  if (failures) fprintf(stderr, "%d failure(s)\n", failures);
  return failures ? 1 : 0;
}
