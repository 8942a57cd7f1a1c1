// Where the keys of selected pages lie (fa_decode.cuh), on the host and under the sanitizers: "page_size max_pages at sel[0] sel[1]
// ..." a line in, with the entries that may be read; the key's position out.
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "../flash_attention_backward_gb300/csrc/fa_decode.cuh"

int main() {
  for (std::string line; std::getline(std::cin, line);) {
    std::istringstream in(line);
    int at;
    fap::Cache c{};
    in >> c.page_size >> c.max_pages >> at;
    fap::page_divisor(c.page_size, &c.page_mul, &c.page_shift);
    std::vector<int32_t> sel;
    for (long long x; in >> x;) sel.push_back((int32_t)x);
    sel.shrink_to_fit();
    std::printf("%d\n", fap::selected_position(c, sel.data(), (int)sel.size() * c.page_size, at));
  }
}
