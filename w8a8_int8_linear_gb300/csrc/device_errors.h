// The device error words of all translation units, as one.
#pragma once
#include <cstddef>

namespace w8a8 {

// Calls every reader (each reads and clears one word; nonzero: it failed), so
// that no word is left to a later query, and puts the first word that is set into
// *code.  Returns the first failure.
template <typename Error, size_t N>
Error read_device_errors(Error (*const (&readers)[N])(unsigned int*), unsigned int* code) {
    *code = 0;
    Error first{};
    for (const auto read : readers) {
        unsigned int word = 0;
        const Error e = read(&word);
        if (first == Error{}) first = e;
        if (e == Error{} && *code == 0) *code = word;
    }
    return first;
}

}  // namespace w8a8
