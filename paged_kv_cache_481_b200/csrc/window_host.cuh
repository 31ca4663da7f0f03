// Host-side checks and dispatch shared by the entry points of pa_window.h.
#pragma once

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

// f(std::true_type) or f(std::false_type): a run-time choice as a template argument.
template <typename F>
auto with_bool(bool b, F &&f)
{
    return b ? f(std::true_type{}) : f(std::false_type{});
}

} // namespace
