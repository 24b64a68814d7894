// Host replay of the 8-bit linear layer's launches (built host-only by
// test_linear8_launches.py; no GPU is needed and no kernel runs).
//
// The program stands in for the few runtime functions that the library calls:
// it reports a gfx950 device, notes every kernel that the library registers
// and, instead of launching one, replays from its arguments the addresses that
// its threads form.  Operands and workspaces are ranges of made-up addresses
// with their exact extents, so an access outside of all of them is found, and
// so is an offset that does not fit the 32 bits the kernels keep it in.  The
// expressions mirror gemm_nt.h, gemm_codes.h and linear8.hip.
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

#include "../post_pruning_amd/csrc/gemm_nt.h"

using sg::NtArgs;
using sg::NtWide;

// ---------------------------------------------------------------------------
// Made-up memory
// ---------------------------------------------------------------------------
namespace {

struct Range {
  const char* name;
  uint64_t at, bytes;
};
std::vector<Range> ranges;
int failures = 0;
std::string what;  // the call being replayed
std::string kernel;

void fail(const char* fmt, ...) {
  if (++failures > 10) return;
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  fprintf(stderr, "FAIL %s: %s: %s\n", what.c_str(), kernel.substr(0, 70).c_str(), buf);
}

template <typename T = void>
T* make(const char* name, uint64_t bytes, uint64_t shift = 0) {
  const uint64_t at = ((uint64_t)ranges.size() + 1) << 56;
  ranges.push_back({name, at + shift, bytes});
  return reinterpret_cast<T*>(at + shift);
}

void touch(const char* who, uint64_t at, uint64_t bytes) {
  for (const Range& r : ranges)
    if (at >= r.at && at + bytes <= r.at + r.bytes) return;
  const uint64_t k = at >> 56;
  if (k >= 1 && k <= ranges.size())
    fail("%s: byte %lld of '%s', which has %lld", who, (long long)(at - ranges[k - 1].at), ranges[k - 1].name,
         (long long)ranges[k - 1].bytes);
  else
    fail("%s: address %llx is in no operand", who, (unsigned long long)at);
}
template <typename T>
uint64_t addr(const T* p) {
  return reinterpret_cast<uint64_t>(p);
}

// An offset that a kernel keeps in 32 bits.
uint64_t in32(const char* who, int64_t off) {
  if (off < 0 || off >= (int64_t)1 << 32) fail("%s: offset %lld does not fit 32 bits", who, (long long)off);
  return (uint32_t)off;
}

void lds(const char* who, int64_t at, int64_t bytes, int64_t size) {
  if (at < 0 || at + bytes > size) fail("%s: LDS bytes %lld + %lld of %lld", who, (long long)at, (long long)bytes, (long long)size);
}

// The first, the last and a few indices between them.
std::vector<int64_t> some(int64_t n) {
  std::set<int64_t> s;
  for (int64_t i : {(int64_t)0, (int64_t)1, n / 2, n - 2, n - 1})
    if (i >= 0 && i < n) s.insert(i);
  return {s.begin(), s.end()};
}
std::vector<int> stages(int n, int ring) {
  std::set<int> s;
  for (int i = 0; i < n && i <= ring; ++i) s.insert(i);
  for (int i = std::max(0, n - ring - 3); i < n; ++i) s.insert(i);
  return {s.begin(), s.end()};
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
struct Tile {
  bool code, i8, bt, offset;
  int TA, TB, WA, WB, RA, RB;
  int waves() const { return WA * WB; }
  int threads() const { return 64 * waves(); }
  int FA() const { return TA / WA / 16; }
  int FB() const { return TB / WB / 16; }
  int GA() const { return FA() / 4; }
};

// The bytes of B's panel: NtPanelB::init and copy.
void panel_b(const Tile& t, const NtArgs& g, int64_t b0, int s0, int n, bool half) {
  const int copies = t.TB / 8 / t.waves();
  const int64_t k0 = (int64_t)s0 * 64;
  const uint64_t base = t.bt ? addr(g.B) + k0 * g.ldb : addr(g.B) + b0 * g.ldb + (int64_t)s0 * 128;
  for (int tid = 0; tid < t.threads(); ++tid) {
    const int wave = tid / 64, lane = tid % 64;
    for (int k = 0; k < copies; ++k) {
      const int r = t.bt ? ((wave * copies + k) * 64 + lane) / (t.TB / 8) : (wave * copies + k) * 8 + (lane >> 3);
      const int piece = (lane & 7) ^ ((r >> 1) & 7);
      int64_t off;
      if (t.bt) {
        const int tau = t.TB == 64 ? ((r >> 1) & 1) | ((r & 8) >> 2) : (r & 3) | ((r & 8) >> 1);
        const int64_t col = b0 + 8 * ((((wave * copies + k) * 64 + lane) % (t.TB / 8)) ^ (2 * tau));
        off = r * g.ldb + 2 * (col + 8 <= g.bcols ? col : g.bcols - 8);
      } else {
        off = std::min<int64_t>(r, g.nb - b0 - 1) * g.ldb + piece * 16;
      }
      in32("B's offset", off);
      for (int s : stages(n, t.RB)) {
        int64_t o = off;
        if (s == n - 1) {
          if (t.bt) {
            const int64_t past = k0 + (int64_t)s * 64 + r - (g.krows - 1);
            if (past > 0) o -= past * g.ldb;
          } else if (half && piece >= 4) {
            o -= 64;
          }
        }
        touch("B", base + (t.bt ? (int64_t)s * 64 * g.ldb : (int64_t)s * 128) + in32("B's offset", o), 16);
      }
      lds("B's copy", (wave * copies + k) * 1024 + lane * 16, 16, t.TB * 128);
    }
  }
}

// NtTile::run
void rows_tile(const Tile& t, const NtArgs& g, int64_t a0, int64_t b0, int s0, int t1) {
  const int n = (t1 + 1) / 2 - s0;
  if (n <= 0) return;
  const bool half = t1 & 1;
  panel_b(t, g, b0, s0, n, half);
  const int ca = t.TA / 8 / t.waves();
  const uint64_t base = addr(g.A) + a0 * g.lda + (int64_t)s0 * 128;
  for (int tid = 0; tid < t.threads(); ++tid) {
    const int wave = tid / 64, lane = tid % 64;
    for (int k = 0; k < ca; ++k) {
      const int64_t r = (wave * ca + k) * 8 + (lane >> 3);
      const int piece = (lane & 7) ^ (2 * (((int)r >> 4) & 3) + (((int)r >> 1) & 1));
      const int64_t off = std::min<int64_t>(r, g.na - a0 - 1) * g.lda + piece * 16;
      in32("A's offset", off);
      for (int s : stages(n, t.RA))
        touch("A", base + (int64_t)s * 128 + in32("A's offset", off - (half && s == n - 1 && piece >= 4 ? 64 : 0)), 16);
      lds("A's copy", (wave * ca + k) * 1024 + lane * 16, 16, t.TA * 128);
    }
  }
}

// CodeTile::run
void code_tile(const Tile& t, const NtArgs& g, int64_t a0, int64_t b0, int s0, int t1) {
  const int n = (t1 + 1) / 2 - s0;
  if (n <= 0) return;
  panel_b(t, g, b0, s0, n, t1 & 1);
  const int64_t k0 = (int64_t)s0 * 64, wide = (g.na + 63) / 64 * 64;
  const uint64_t base = addr(g.A) + k0 * g.lda;
  for (int tid = 0; tid < t.threads(); ++tid) {
    const int kr = tid / (t.TA / 16), p = tid % (t.TA / 16);
    const int64_t off = kr * g.lda + std::min<int64_t>(a0 + 16 * p, wide - 16);
    in32("A's offset", off);
    for (int s : stages(n, t.RB)) {
      int64_t past = 0;
      if (s == n - 1) past = std::max<int64_t>(0, k0 + (int64_t)s * 64 + kr - (g.krows - 1));
      touch("A's codes", base + (int64_t)s * 64 * g.lda + in32("A's offset", off - past * g.lda), 16);
      touch("A's scales", addr(g.k_scale + k0) + (int64_t)s * 256 + in32("the scales' offset", (kr - past) * 4), 4);
      if (t.offset)
        touch("A's offsets", addr(g.k_off + k0) + (int64_t)s * 256 + in32("the offsets' offset", (kr - past) * 4), 4);
    }
    lds("A's copy", tid * 16, 16, t.TA * 64);
  }
}

// What one wave's corner stores of fragment j: 64 columns, 16 rows.
void outputs(const NtArgs& g, int64_t a0, int64_t b0, bool masked, const NtWide& wide) {
  const int64_t e = g.out_dtype == SG_F32 ? 4 : 2;
  const bool aligned = wide.out4 && (!masked || !g.mask || wide.mask16 || wide.mask4);
  for (int lane = 0; lane < 64; ++lane) {
    if (aligned) {
      const int64_t a = a0 + (lane >> 4) * 16, b = b0 + (lane & 15);
      if (b >= g.nb || a >= g.na) continue;
      const int64_t cnt = std::min<int64_t>(g.na - a, 16);
      touch("out", addr(static_cast<char*>(g.out)) + (b * g.ldo + a) * e, cnt * e);
      if (masked && g.mask) touch("mask", addr(g.mask) + b * g.na + a, cnt);
      if (g.a_scale) touch("a_scale", addr(g.a_scale + a), 4 * cnt);
      if (g.a_off) touch("a_off", addr(g.a_off + a), 4 * cnt);
      if (g.b_scale) touch("b_scale", addr(g.b_scale + b), 4);
      if (g.b_sum) touch("b_sum", addr(g.b_sum + b), 4);
    } else {
      const int64_t a = a0 + lane;
      if (a0 >= g.na || b0 >= g.nb || a >= g.na) continue;
      for (int64_t r = 0; r < std::min<int64_t>(16, g.nb - b0); ++r) {
        touch("out", addr(static_cast<char*>(g.out)) + ((b0 + r) * g.ldo + a) * e, e);
        if (masked && g.mask) touch("mask", addr(g.mask) + (b0 + r) * g.na + a, 1);
        if (g.b_scale) touch("b_scale", addr(g.b_scale + b0 + r), 4);
        if (g.b_sum) touch("b_sum", addr(g.b_sum + b0 + r), 4);
      }
      if (g.a_scale) touch("a_scale", addr(g.a_scale + a), 4);
      if (g.a_off) touch("a_off", addr(g.a_off + a), 4);
    }
  }
}

void all_outputs(const Tile& t, const NtArgs& g, int64_t a0, int64_t b0, bool masked, const NtWide& wide) {
  for (int wave = 0; wave < t.waves(); ++wave)
    for (int h = 0; h < t.GA(); ++h)
      for (int j = 0; j < t.FB(); ++j)
        outputs(g, a0 + (wave / t.WB) * (t.TA / t.WA) + h * 64, b0 + (wave % t.WB) * (t.TB / t.WB) + j * 16, masked, wide);
}

bool parse_tile(const std::string& name, Tile& t, int& ep, bool& split) {
  std::vector<std::string> v;
  const size_t at = name.find("Tile<");
  if (at == std::string::npos) return false;
  t = Tile{};
  t.code = name.compare(at - 4, 4, "Code") == 0;
  std::string word;
  for (size_t i = at + 5; i < name.size() && name[i] != '('; ++i) {
    const char c = name[i];
    if (c == ',' || c == '>') {
      if (!word.empty()) v.push_back(word);
      word.clear();
    } else if (c != ' ') {
      word += c;
    }
  }
  auto num = [&](size_t i) { return i < v.size() ? (v[i] == "true" ? 1 : v[i] == "false" ? 0 : atoi(v[i].c_str())) : 0; };
  size_t i = 0;
  if (!t.code) t.i8 = num(i++);
  t.TA = num(i++), t.TB = num(i++), t.WA = num(i++), t.WB = num(i++);
  t.RA = t.code ? 0 : num(i++);
  t.RB = num(i++);
  t.bt = num(i++);
  if (t.code) t.offset = num(i++);
  ep = num(i++);
  split = num(i++);
  return t.TA > 0 && t.TB > 0 && t.WA > 0 && t.WB > 0 && t.RB > 0;
}

// ---------------------------------------------------------------------------
// Kernels
// ---------------------------------------------------------------------------
std::map<std::string, int> seen;  // launches of each kernel
int64_t rows_done;                // of the call's output, in launches that follow each other

// A launch that takes rows [first, first + rows) of what starts at `base`.
void next_rows(uint64_t at, uint64_t base, int64_t pitch, int64_t rows) {
  if (rows < 1 || at != base + rows_done * pitch) fail("rows left out after %lld", (long long)rows_done);
  rows_done += rows;
}

template <typename T>
const T& arg(void** a, int i) {
  return *static_cast<const T*>(a[i]);
}

struct PadRows {  // as in linear8.hip
  uint16_t* dst;
  int64_t pitch;
  const uint16_t* src;
  int64_t lds, rows, cols;
};

void replay_tile(void** a, dim3 grid, dim3 block) {
  Tile t;
  int ep;
  bool split;
  if (!parse_tile(kernel, t, ep, split)) return fail("name not understood");
  const NtArgs& g = arg<NtArgs>(a, 0);
  const NtWide& wide = arg<NtWide>(a, 1);
  const int64_t ta = arg<int64_t>(a, 2), tb = arg<int64_t>(a, 3);
  const int splits = arg<int>(a, 4);
  char* const part = arg<char*>(a, 5);
  if ((int)block.x != t.threads()) fail("%u threads", block.x);
  if (ta != sg::ceil_div(g.na, t.TA) || tb != sg::ceil_div(g.nb, t.TB)) fail("%lld x %lld tiles", (long long)ta, (long long)tb);
  if ((int64_t)grid.x < ta * tb * splits) fail("%u workgroups", grid.x);
  next_rows(addr(static_cast<char*>(g.out)), ranges[0].at, g.ldo * (g.out_dtype == SG_F32 ? 4 : 2), g.nb);
  const int steps = (int)(g.kbytes / 64), nst = (steps + 1) / 2;
  for (int64_t ia : some(ta))
    for (int64_t ib : some(tb))
      for (int64_t sp : some(splits)) {
        int s0 = 0, t1 = steps;
        if (split) {
          s0 = (int)((int64_t)nst * sp / splits);
          t1 = std::min(steps, 2 * (int)((int64_t)nst * (sp + 1) / splits));
        }
        (t.code ? code_tile : rows_tile)(t, g, ia * t.TA, ib * t.TB, s0, t1);
        const int64_t slots = (int64_t)t.FA() * t.FB() * t.threads();
        if (split)  // the tile's number takes every value below ta tb
          for (int64_t k : {(int64_t)0, ta * tb - 1}) touch("partial sums", addr(part) + (k * splits + sp) * slots * 16, slots * 16);
        else
          all_outputs(t, g, ia * t.TA, ib * t.TB, ep == sg::EP_MASKED, wide);
      }
}

void replay_join(void** a, dim3 grid, dim3 block) {
  Tile t;
  int ep;
  bool split;
  if (!parse_tile(kernel, t, ep, split)) return fail("name not understood");
  const NtArgs& g = arg<NtArgs>(a, 0);
  const int64_t ta = arg<int64_t>(a, 2), tb = arg<int64_t>(a, 3);
  const int splits = arg<int>(a, 4);
  if ((int64_t)grid.x != ta * tb || (int)grid.y != t.GA() * t.FB() || (int)block.x != t.threads()) fail("launch shape");
  const int64_t slots = (int64_t)t.FA() * t.FB() * t.threads();
  touch("partial sums", addr(arg<char*>(a, 5)), ta * tb * splits * slots * 16);
  for (int64_t ia : some(ta))
    for (int64_t ib : some(tb)) all_outputs(t, g, ia * t.TA, ib * t.TB, ep == sg::EP_MASKED, arg<NtWide>(a, 1));
}

void replay_stream(void** a, dim3 grid, dim3 block) {
  const NtArgs& g = arg<NtArgs>(a, 0);
  // <I8, EP, CF, TF, W, U>
  const size_t at = kernel.find("nt_stream_kernel<");
  int v[6] = {0}, k = 0;
  std::string word;
  for (size_t i = at + 17; k < 6 && i < kernel.size(); ++i) {
    if (kernel[i] == ',' || kernel[i] == '>') {
      v[k++] = word == "true" ? 1 : atoi(word.c_str());
      word.clear();
    } else if (kernel[i] != ' ') {
      word += kernel[i];
    }
  }
  const int CF = v[2], TF = v[3], W = v[4];
  next_rows(addr(static_cast<char*>(g.out)), ranges[0].at, 0, g.nb);
  if ((int)block.x != 64 * W || (int64_t)grid.x != sg::ceil_div(g.na, 16 * CF) || g.nb > 16 * TF) fail("launch shape");
  const int steps = (int)(g.kbytes / 64);
  for (int64_t wg : some(grid.x))
    for (int wave = 0; wave < W; ++wave) {
      const int s0 = steps * wave / W, s1 = steps * (wave + 1) / W;
      if (s0 == s1) continue;
      for (int lane = 0; lane < 64; ++lane) {
        const int64_t bytes = (int64_t)(s1 - 1 - s0) * 64 + 16;
        for (int c = 0; c < CF; ++c)
          touch("A", addr(g.A) + std::min<int64_t>(wg * 16 * CF + 16 * c + (lane & 15), g.na - 1) * g.lda + (lane >> 4) * 16 +
                         (int64_t)s0 * 64, bytes);
        for (int f = 0; f < TF; ++f)
          touch("B", addr(g.B) + std::min<int64_t>(16 * f + (lane & 15), g.nb - 1) * g.ldb + (lane >> 4) * 16 + (int64_t)s0 * 64,
                bytes);
      }
    }
}

void replay_operands(void** a, dim3 grid, dim3) {
  uint16_t* const wt = arg<uint16_t*>(a, 0);
  const int64_t Rp = arg<int64_t>(a, 1);
  const int8_t* const codes = arg<int8_t*>(a, 2);
  const int64_t ldc = arg<int64_t>(a, 3);
  const float* const scale = arg<float*>(a, 4);
  const int32_t* const offset = arg<int32_t*>(a, 5);
  const int64_t R = arg<int64_t>(a, 6), C = arg<int64_t>(a, 7), tblocks = arg<int64_t>(a, 8);
  const PadRows pad = arg<PadRows>(a, 9);
  if ((int64_t)grid.x > tblocks) {
    const int64_t cpr = pad.pitch / 8;
    for (int64_t t : some(pad.rows))
      for (int64_t c : some(cpr)) {
        for (int e = 0; e < 8; ++e)
          if (c * 8 + e < pad.cols) touch("the rows to pad", addr(pad.src + t * pad.lds + c * 8 + e), 2);
        touch("the padded rows", addr(pad.dst + t * pad.pitch + c * 8), 16);
      }
  }
  if (tblocks == 0) return;
  const int64_t tc = (C + 63) / 64, tr = (Rp + 63) / 64;
  for (int64_t ir : some(tr))
    for (int64_t ic : some(tc))
      for (int tid = 0; tid < 256; ++tid) {
        const int64_t r0 = ir * 64, c0 = ic * 64, r = r0 + (tid >> 2);
        const int lc = (tid & 3) * 16;
        if (r < R && c0 + lc < C) {
          touch("codes", addr(codes + r * ldc + c0 + lc), 16);
          touch("scales", addr(scale + r), 4);
          if (offset) touch("offsets", addr(offset + r), 4);
        }
        for (int k = 0; k < 2; ++k) {
          const int item = tid + 256 * k, c = item >> 3, rr = (item & 7) * 8;
          if (c0 + c < C && r0 + rr < Rp) touch("bf16 rows", addr(wt + (c0 + c) * Rp + r0 + rr), 16);
        }
      }
}

void replay_quantize(void** a, dim3 grid, dim3 block) {
  int8_t* const Q = arg<int8_t*>(a, 0);
  const int64_t ldq = arg<int64_t>(a, 1), T = arg<int64_t>(a, 5), n = arg<int64_t>(a, 6), ldx = arg<int64_t>(a, 7);
  const char* const X = arg<char*>(a, 4);
  const int64_t e = kernel.find("quantize_kernel<float") != std::string::npos ? 4 : 2;
  const int tpr = atoi(kernel.c_str() + kernel.find(',') + 1);
  if ((int64_t)grid.x * block.x < T * tpr || (int)block.x < tpr) fail("%u x %u threads", grid.x, block.x);
  if (tpr > 64 && ((int64_t)grid.x != T || (int)block.x != tpr)) fail("rows behind the last");
  next_rows(addr(Q), ranges[0].at, ldq, T);
  for (int64_t t : some(T)) {
    touch("X", addr(X) + t * ldx * e, n * e);
    touch("Q", addr(Q + t * ldq), sg::round_up(n, 64));
    touch("scale", addr(arg<float*>(a, 2) + t), 4);
    touch("sum", addr(arg<int32_t*>(a, 3) + t), 4);
  }
}

void replay_dequantize(void** a, dim3 grid, dim3 block) {
  const char* const X = arg<char*>(a, 0);
  const int64_t ldx = arg<int64_t>(a, 1), ldq = arg<int64_t>(a, 3), T = arg<int64_t>(a, 5), n = arg<int64_t>(a, 6);
  const int64_t e = kernel.find("dequantize_kernel<float") != std::string::npos ? 4 : 2;
  if ((int64_t)grid.x * block.x * 16 < n || block.x * block.y != 256) fail("launch shape");
  next_rows(addr(X), ranges[0].at, 0, T);
  for (int64_t t : some(T)) {
    touch("X", addr(X) + t * ldx * e, n * e);
    touch("Q", addr(arg<int8_t*>(a, 2) + t * ldq), sg::round_up(n, 16));
    touch("scale", addr(arg<float*>(a, 4) + t), 4);
  }
}

void replay(void** a, dim3 grid, dim3 block) {
  // what a launch may have: less than 2^32 threads in each direction
  for (uint64_t threads : {(uint64_t)grid.x * block.x, (uint64_t)grid.y * block.y, (uint64_t)grid.z * block.z})
    if (threads < 1 || threads >= (uint64_t)1 << 32) fail("%llu threads", (unsigned long long)threads);
  if (grid.y > 65535 || grid.z > 65535 || block.x * block.y * block.z > 1024) fail("launch shape");
  const auto is = [](const char* s) { return kernel.find(s) != std::string::npos; };
  if (is("nt_tile_kernel"))
    replay_tile(a, grid, block);
  else if (is("nt_join_kernel"))
    replay_join(a, grid, block);
  else if (is("nt_stream_kernel"))
    replay_stream(a, grid, block);
  else if (is("operands_kernel"))
    replay_operands(a, grid, block);
  else if (is("::quantize_kernel"))
    replay_quantize(a, grid, block);
  else if (is("::dequantize_kernel"))
    replay_dequantize(a, grid, block);
  else
    fail("unknown kernel");
}

// (the library registers its kernels before this program's own objects exist)
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

// ---------------------------------------------------------------------------
// The runtime's functions that the library calls
// ---------------------------------------------------------------------------
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

// A call that succeeded has taken every row of its output, its first operand here.
void expect_ok(sg_status s, int64_t rows) {
  if (s != SG_OK) fail("status %d: %s", (int)s, sg_last_error_message());
  if (rows_done != rows) fail("%lld of %lld rows", (long long)rows_done, (long long)rows);
}
void begin(const char* call, int64_t T, int64_t n, int64_t m) {
  ranges.clear();
  rows_done = 0;
  kernel = "-";
  char buf[200];
  snprintf(buf, sizeof(buf), "%s T=%lld n=%lld m=%lld", call, (long long)T, (long long)n, (long long)m);
  what = buf;
}

// Operands exactly as large as the interface asks for.
struct Rows {
  void* p;
  int64_t ld;
};
Rows codes(const char* name, int64_t rows, int64_t n, int64_t extra = 0) {
  const int64_t pad = sg::round_up(n, SG_CODE_PITCH), ld = pad + extra;
  return {make(name, rows > 0 ? (rows - 1) * ld + pad : 0), ld};
}
Rows values(const char* name, int64_t rows, int64_t cols, int64_t e, int64_t extra = 0, int64_t shift = 0) {
  const int64_t ld = cols + extra;
  return {make(name, rows > 0 ? ((rows - 1) * ld + cols) * e : 0, shift * e), ld};
}

void linear(int64_t T, int64_t n, int64_t m, int dtype, int64_t extra = 0, int64_t shift = 0, int64_t code = 0) {
  begin("linear", T, n, m);
  const int64_t e = dtype == SG_F32 ? 4 : 2;
  const Rows y = values("Y", T, m, e, extra, shift), q = codes("Q", T, n, code), w = codes("Wq", m, n, code);
  const size_t nb = sg_workspace_bytes(SG_OP_LINEAR_W8A8, m, n, T, 0);
  expect_ok(sg_linear_w8a8(y.p, dtype, y.ld, (int8_t*)q.p, q.ld, make<float>("x_scale", 4 * T), make<int32_t>("x_sum", 4 * T), T,
                           (int8_t*)w.p, w.ld, make<int32_t>("w_offset", 4 * m), make<float>("w_scale", 4 * m), m, n,
                           make("workspace", nb), nb, nullptr),
            T);
}

void grad_input(int64_t T, int64_t n, int64_t m, int dtype, int64_t extra = 0, int64_t shift = 0, int64_t code = 0,
                int64_t out = -1) {
  begin("grad_input", T, n, m);
  const int64_t e = dtype == SG_F32 ? 4 : 2;
  const Rows dx = values("dX", T, n, e, out < 0 ? extra : out, shift), dy = values("dY", T, m, 2, extra, shift),
             w = codes("Wq", m, n, code);
  const size_t nb = sg_workspace_bytes(SG_OP_GRAD_INPUT, m, n, T, 0);
  expect_ok(sg_linear_w8_grad_input(dx.p, dtype, dx.ld, dy.p, SG_BF16, dy.ld, T, (int8_t*)w.p, w.ld,
                                    make<int32_t>("w_offset", 4 * m), make<float>("w_scale", 4 * m), m, n,
                                    make("workspace", nb), nb, nullptr),
            T);
}

void grad_weight(int64_t T, int64_t n, int64_t m, int dtype, int64_t extra = 0, int64_t shift = 0, int64_t code = 0,
                 int64_t out = -1) {
  begin("grad_weight", T, n, m);
  const int64_t e = dtype == SG_F32 ? 4 : 2;
  const Rows dw = values("dW", m, n, e, out < 0 ? extra : out, shift), dy = values("dY", T, m, 2, extra, shift),
             q = codes("Q", T, n, code);
  const size_t nb = sg_workspace_bytes(SG_OP_GRAD_WEIGHT, m, n, T, 0);
  uint8_t* const mask = make<uint8_t>("mask", m * n);
  expect_ok(sg_linear_w8_grad_weight(dw.p, dtype, dw.ld, 0, dy.p, SG_BF16, dy.ld, (int8_t*)q.p, q.ld,
                                     make<float>("x_scale", 4 * T), T, mask, m, n, make("workspace", nb), nb, nullptr),
            m);
}

void checkpoint(int64_t T, int64_t n, int dtype, int64_t extra = 0, int64_t shift = 0) {
  const int64_t e = dtype == SG_F32 ? 4 : 2;
  begin("quantize", T, n, 0);
  Rows q = codes("Q", T, n), x = values("X", T, n, e, extra, shift);
  expect_ok(sg_quantize_tokens((int8_t*)q.p, q.ld, make<float>("scale", 4 * T), make<int32_t>("sum", 4 * T), x.p, dtype, T, n,
                               x.ld, nullptr),
            T);
  begin("dequantize", T, n, 0);
  x = values("X", T, n, e, extra, shift), q = codes("Q", T, n);
  expect_ok(sg_dequantize_tokens(x.p, dtype, x.ld, (int8_t*)q.p, q.ld, make<float>("scale", 4 * T), T, n, nullptr), T);
}

typedef std::vector<std::vector<int64_t>> Sizes;

// Shapes that between them reach every tile, whole and split, with rows of
// every alignment.
const Sizes kShapes = {
    {1, 1, 1}, {33, 33, 33}, {70, 33, 8200}, {70, 4100, 33}, {33, 8200, 4100}, {70, 33000, 4100}, {300, 130, 9000},
    {2303, 200, 2001}, {5, 130, 131077}, {20001, 130, 70}, {203, 8200, 20001}, {8200, 70, 770}, {2050, 70, 4100},
    {33, 2050, 4100}, {70, 20001, 33}, {3301, 3295, 100}, {20001, 203, 8200}, {8200, 203, 4100}, {770, 70, 8200},
    {4100, 70, 2050}, {770, 33, 33}, {4100, 2050, 70}, {33, 130, 131077}, {515, 1000, 770}, {9000, 132, 70},
    {129, 1000, 2050}, {20001, 8200, 203}, {512, 4096, 4096}, {8192, 4096, 11008}, {64, 4096, 4096}, {130, 33000, 33}};

void shapes() {
  for (const auto& s : kShapes)
    for (int dtype : {SG_F32, SG_BF16})
      for (int64_t extra : {0, 4, 3})
        for (int64_t shift : {0, 1}) {
          linear(s[0], s[1], s[2], dtype, extra, shift);
          grad_input(s[0], s[1], s[2], dtype, extra, shift);
          grad_weight(s[0], s[1], s[2], dtype, extra, shift);
          checkpoint(s[0], s[1], dtype, extra, shift);
        }
}

// Rows as far apart as the interface allows.
void pitches() {
  const int64_t far = (int64_t)1 << 23;
  for (const auto& s : kShapes) {
    const int64_t T = s[0], n = s[1], m = s[2], code = far - sg::round_up(n, SG_CODE_PITCH);
    linear(T, n, m, SG_F32, far / 4 - m, 0, code);
    linear(T, n, m, SG_BF16, far / 2 - m, 1, code);
    grad_input(T, n, m, SG_F32, far / 2 - m, 0, code, far / 4 - n);
    grad_input(T, n, m, SG_BF16, far / 2 - 1 - m, 1, code, far / 2 - n);
    grad_weight(T, n, m, SG_F32, far / 2 - m, 0, code, far / 4 - n);
    grad_weight(T, n, m, SG_BF16, far / 2 - 1 - m, 1, code, far / 2 - n);
  }
}

// Up to the largest sizes that the interface allows.
void weight_gradient_of_many_tokens() {
  const int64_t top = ((int64_t)1 << 31) - 1;
  for (int64_t T : {(int64_t)4000000, (int64_t)8388608, (int64_t)8388609, (int64_t)8421504, (int64_t)8421505, (int64_t)9000000,
                    (int64_t)16900000, (int64_t)17000000, (int64_t)34000000, (int64_t)34100000, (int64_t)100000000, top})
    for (int64_t n : {33, 128, 512, 1000, 1024, 4096, 65536})
      for (int64_t m : {33, 128, 512, 1000, 2048, 11008, 1 << 20}) grad_weight(T, n, m, SG_F32);
}

// More rows than one launch takes.
void many_tokens() {
  for (int64_t T : {((int64_t)1 << 22) + 3, ((int64_t)1 << 24) + 3, ((int64_t)1 << 26) + 3, ((int64_t)1 << 29) + 70,
                    ((int64_t)1 << 30) + 70, ((int64_t)1 << 31) - 1}) {
    for (int64_t n : {1, 100, 1024, 1025, 8192, 8193, 32768, 32769, 65536})
      for (int dtype : {SG_F32, SG_BF16}) checkpoint(T, n, dtype);
    for (int64_t n : {1, 64, 65, 1000, 65536})
      for (int64_t m : {1, 64, 65, 129, 1000, 1 << 20}) {
        // (2^39 outputs are four times the card's memory)
        if (T * m <= (int64_t)1 << 39) linear(T, n, m, SG_BF16);
        if (T * n <= (int64_t)1 << 39) grad_input(T, n, m, SG_BF16);
      }
  }
  // and many output channels
  for (int64_t T : {1, 70, 700, 70000})
    for (int64_t n : {1, 64, 1000, 65536}) {
      linear(T, n, 1 << 20, SG_F32);
      grad_input(T, n, 1 << 20, SG_F32);
      grad_weight(T, n, 1 << 20, SG_F32);
    }
}

}  // namespace

int main(int argc, char** argv) {
  const std::string test = argc > 1 ? argv[1] : "";
  if (test == "shapes")
    shapes();
  else if (test == "pitches")
    pitches();
  else if (test == "many_tokens")
    many_tokens();
  else if (test == "weight_gradient_of_many_tokens")
    weight_gradient_of_many_tokens();
  else
    return 2;
  int total = 0;
  for (const auto& s : seen) {
    printf("%6d %s\n", s.second, s.first.c_str());
    total += s.second;
  }
  if (failures) {
    fprintf(stderr, "%d failure(s)\n", failures);
    return 1;
  }
  printf("%d launches replayed\n", total);
  return total ? 0 : 3;
}
