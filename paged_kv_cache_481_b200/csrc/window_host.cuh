// Host-side checks and dispatch shared by the entry points of pa_window.h.
#pragma once

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/pa_window.h"

namespace {

bool valid_dtype(int t)
{
    return t == PA_F16 || t == PA_BF16;
}

bool valid_kv8(int t)
{
    return t == PA_KV8_INT8 || t == PA_KV8_E4M3;
}

// num_heads a whole multiple of num_kv_heads, at most 128 query heads each
bool valid_heads(int num_heads, int num_kv_heads)
{
    return num_heads > 0 && num_kv_heads > 0 && num_heads <= 65535 &&
           num_heads % num_kv_heads == 0 && num_heads / num_kv_heads <= 128;
}

// Heads of one block's row of scales (rounded up to even: 16-byte rows).
int scale_heads(int num_kv_heads)
{
    return num_kv_heads + (num_kv_heads & 1);
}

// Weights enter the product with V 2^shift times the softmax's, up to 2^8 more
// with a stale reference, and are summed unnormalised.  fp16 weights are made
// larger, 2^7, so that those down to 2^-31 of the largest count.  bf16 ones
// have the range of fp32, and so has V: they are made so small that all the
// tokens a query sees weigh at most 1 together, and a sum of finite V rows
// stays finite.  (At the other end, V below 2^-133 times their number loses
// bits to fp32's smallest step.)
float weight_shift(bool bf16, int max_context_len, int window, int num_sinks)
{
    if (!bf16)
        return 7.0f;
    const int64_t seen = std::min(int64_t(max_context_len), int64_t(window) + num_sinks);
    int bits = 0;
    while ((int64_t(1) << bits) < seen)
        ++bits;
    return float(-8 - bits);
}

// f(std::true_type) or f(std::false_type): a run-time choice as a template argument.
template <typename F>
auto with_bool(bool b, F &&f)
{
    return b ? f(std::true_type{}) : f(std::false_type{});
}

} // namespace
