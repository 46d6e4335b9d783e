// moe_tree_attention8: which kernel takes a call, for one kind of codes (a translation unit each).
#pragma once

#include "moe_tree_attn.cuh"

namespace moe {

int attention8_i8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream);

namespace {

// Query rows a key/value head up to which products of codes are taken in registers (moe_few_rows.cuh), and
// above which through tensor memory.  16 requests over 4,096 to 8,192 keys in blocks of 64, 8 query heads a
// key/value head, us in registers / through tensor memory:
//   query rows       8        16        24 and 32    48         64
//   8 heads of 64    41 / 76  47 / 77   64 / 77      112 / 78   112 / 78    e4m3
//                    43 / 80  48 / 82   65 / 82      113 / 84   114 / 84    int8
//   4 heads of 128   33 / 57  39 / 57   55 / 58      86 / 59    86 / 59     e4m3
//                    35 / 65  41 / 65   56 / 65      88 / 67    88 / 67     int8
//   2 heads of 256   35 / 55  42 / 55   60 / 57      81 / 62    99 / 64     e4m3
//                    36 / 63  41 / 64   61 / 64      84 / 69    104 / 70    int8
// (Heads of 256 have 16 rows a group there, so 17 to 32 read the keys twice: 5 % slower than through tensor memory
// with e4m3, 4 % faster with int8.)  The kernel goes by max_tree, not by the rows that a request brings.
constexpr int kFewRows = 32;

template <int FMT>
int choose(const moe_tree_attention8_args& a, const Plan& p, int sms, cudaStream_t st) {
  using A = moe_tree_attention8_args;
  // Few query rows a head: products of codes in registers, in groups of up to 32 query rows (heads of 256: 16).
  const int rows = a.max_tree * p.group, nt = rows > kFewRows ? 0 : rows <= 8 ? 1 : rows <= 16 || a.head_dim == 256 ? 2 : 4;
  using I = std::integral_constant<int, 64>;
  using J = std::integral_constant<int, 128>;
  using K = std::integral_constant<int, 256>;
  if (nt) {
    const auto few = [&](auto d, auto n) { return launch<A, FMT, decltype(d)::value, 0, decltype(n)::value>(a, p, sms, st); };
    std::integral_constant<int, 1> one;
    std::integral_constant<int, 2> two;
    std::integral_constant<int, 4> four;
    if (a.head_dim == 64) return nt == 1 ? few(I{}, one) : nt == 2 ? few(I{}, two) : few(I{}, four);
    if (a.head_dim == 128) return nt == 1 ? few(J{}, one) : nt == 2 ? few(J{}, two) : few(J{}, four);
    return nt == 1 ? few(K{}, one) : few(K{}, two);
  }
  // Blocks of 16 tokens and more have one scale for each run of 16 keys of a tile, those of 8 for each of 8;
  // smaller ones are taken key by key.
  const auto many = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return a.cache.block_size >= 16  ? launch<A, FMT, D, 16>(a, p, sms, st)
           : a.cache.block_size == 8 ? launch<A, FMT, D, 8>(a, p, sms, st)
                                     : launch<A, FMT, D, 0>(a, p, sms, st);
  };
  return a.head_dim == 64 ? many(I{}) : a.head_dim == 128 ? many(J{}) : many(K{});
}

template <int FMT>
int attention8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream) {
  Plan p{};
  int sms = 0;
  const int rc = prepare(args, ws, ws_bytes, p, sms);
  if (rc != MOE_OK || args->n_rows == 0) return rc;
  const moe_tree_attention8_args& a = *args;
  p.flip = 0;
  p.c = 1.f;
  p.score = a.scale * 1.4426950408889634f;
  while ((1 << p.block_shift) < a.cache.block_size) ++p.block_shift;
  return choose<FMT>(a, p, sms, static_cast<cudaStream_t>(stream));
}

}  // namespace

}  // namespace moe
